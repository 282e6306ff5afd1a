// sps_dense.hip -- softmax cross entropy of dense queries over dense items, and
// its gradients, without the logits.
//
// With z = x . w / tau + b and G = weight / tau (softmax(z) - onehot(target)):
//   loss = lse(z) - z_target,  grad x = G w,  grad w = G^T x.
// Three matrix products, the least there is, for a piece of the rows at a time:
//   1. logits: a tile's z in registers; its rows' maxima and sums of
//      exponentials go to `stats`, and e^(z - max) in 16 bits to `code`;
//   2. a row's log-sum-exp and loss from its blocks' statistics, and its codes to
//      G in place;
//   3. two products with G: for the queries its k (items) lies in one run, for
//      the items it is read turned.
// Code: a 16-bit float below the block's maximum, so that z is not computed
// twice. It has a bit more than fp16's G and three more than bf16's, down to
// 2^-30 (bf16: 2^-29) of the block's maximum, and runs out gradually below. G's
// own column at the target is 1 - p from the loss, never p - 1 of a rounded p.
// fp16: G is held 2^k times as large, 2^k the power of two that takes the
// largest weight to [2^14, 2^15), so that where p times its row's weight is down
// to 2^-28 of that weight G keeps all its bits.
// float32: operands and G stand in two planes of fp16, scaled by powers of two
// (each row for the logits, the matrix for the products with G, whose sums go
// over rows), so that a value keeps 22 bits down to 2^-17 of the largest and
// an absolute 2^-39 of it below; three products of planes leave out what is
// below 2^-22 of a product. (Three planes of bf16 and six products of them:
// 1000 x 30,522 x 384 605 us instead of 389.)
// Bound by the three products: 8192 x 100,000 x 1024 bf16 takes 5.03 ms, of which
// the logits 1.62 to 1.68 (1.03 to 1.0 PFLOP/s; a library's product of that shape
// 1.34 ms, without exponentials, sums and codes), both other products 2.59 to
// 2.74 (1.29 to 1.22), codes to G 0.70, rows laid out 0.12.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sps_gemm.h"

namespace sps {

// ---------------------------------------------------------------------------
// operands

// 16-bit planes of a value: itself, or a float32 as lead + rest in fp16.
template <typename T>
constexpr int kPlanes = 1;
template <>
constexpr int kPlanes<float> = 2;

__device__ __forceinline__ void split(f16_t x, uint16_t o[1]) { o[0] = x.u; }
__device__ __forceinline__ void split(bf16_t x, uint16_t o[1]) { o[0] = x.u; }
// Infinities and NaN stand in the leading plane.
__device__ __forceinline__ void split(float x, uint16_t o[2]) {
  const f16_t lead = from_f32<f16_t>(x);
  const float h = to_f32(lead);
  o[0] = lead.u;
  o[1] = from_f32<f16_t>(fabsf(h) < __builtin_inff() ? x - h : 0.0f).u;
}
// The power of two that takes a largest magnitude to [2^14, 2^15) (1 for 0; at most 2^127).
__device__ __forceinline__ float scale_for(float top) {
  int e = 14 - ((int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127);
  e = top == 0.0f ? 0 : (e > 127 ? 127 : e);
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}
// And back: scales are divided out by their exponents together, since one of two may leave the
// range where both do not.
__device__ __forceinline__ int exponent_of(float scale) {
  return (int)(__builtin_bit_cast(uint32_t, scale) >> 23) - 127;
}
// fp16 x power of two: the type does not change
template <typename T>
__device__ __forceinline__ T scaled(T x, float) { return x; }
template <>
__device__ __forceinline__ float scaled(float x, float s) { return x * s; }

// Rows that take no part are zeros in the transposed copy, so that what they
// hold (padding, NaN) meets the gradient's zeros as zero: rows of queries
// without a target or weight, items whose bias is -inf.
struct RowMask {
  const int32_t *targets;
  const float *weights;
  int64_t m;
  const float *bias;
  __device__ __forceinline__ bool out(int64_t r) const {
    if (targets) {
      const int32_t t = targets[r];
      return t < 0 || t >= m || (weights && weights[r] == 0.0f);
    }
    return bias && bias[r] == -__builtin_inff();
  }
};

struct LayArgs {
  const void *x;
  int64_t ld, rows, cols;
  uint16_t *packed;  // nullable: [rows][ld_p], zeros from cols on
  int64_t ld_p, plane_p;
  uint16_t *turned;  // nullable: [cols][ld_t], zeros from rows on
  int64_t ld_t, plane_t;
  RowMask mask;
  // float32: the scales, of every row in the packed planes and of all rows that take part in the
  // turned ones (kMaxBlocks partial maxima)
  float *row_scale;
  float *tops;
};
constexpr int kMaxBlocks = 256;

// float32: scales of rows and partial maxima, a wave for kMaxRowsOnce rows; bound
// by memory: 31,522 rows of 384 in 14 us, 3.5 TB/s (a row at a time: 64).
// What is not finite has no part in a scale.
struct MaxBoth {
  LayArgs side[2];
};
constexpr int kMaxWaves = 16, kMaxRowsOnce = 4;
__global__ __launch_bounds__(64 * kMaxWaves) void ce_max_kernel(MaxBoth both) {
  const LayArgs a = blockIdx.x >= kMaxBlocks ? both.side[1] : both.side[0];
  const int block = blockIdx.x % kMaxBlocks, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __shared__ float tops[kMaxWaves];
  const float *const x = static_cast<const float *>(a.x);
  float most = 0.0f;
  // a few rows at a time, so that their loads are on their way together
  for (int64_t r0 = ((int64_t)block * kMaxWaves + wave) * kMaxRowsOnce; r0 < a.rows;
       r0 += kMaxBlocks * kMaxWaves * kMaxRowsOnce) {
    float top[kMaxRowsOnce] = {};
    for (int64_t c = lane; c < a.cols; c += 64)
#pragma unroll
      for (int i = 0; i < kMaxRowsOnce; ++i) {
        const int64_t r = r0 + i < a.rows ? r0 + i : r0;
        const float f = fabsf(x[r * a.ld + c]);
        if (f < __builtin_inff()) top[i] = fmaxf(top[i], f);
      }
#pragma unroll
    for (int i = 0; i < kMaxRowsOnce; ++i) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) top[i] = fmaxf(top[i], __shfl_xor(top[i], o, 64));
      if (r0 + i >= a.rows) continue;
      if (lane == 0) a.row_scale[r0 + i] = scale_for(top[i]);
      if (!a.mask.out(r0 + i)) most = fmaxf(most, top[i]);
    }
  }
  if (lane == 0) tops[wave] = most;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < kMaxWaves; ++i) most = fmaxf(most, tops[i]);
  a.tops[block] = most;
}
// The scale of a turned matrix; every thread of 256 calls it.
__device__ __forceinline__ float turned_scale(const float *parts) {
  __shared__ float tops[4];
  float top = parts[threadIdx.x];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  return scale_for(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
}

// Tiles of 64 x 64 through LDS, 8 values a thread and step both ways; bound by
// memory (30,522 + 4095 rows of 768 in 16 bits turned: 28 us, 3.8 TB/s). Planes
// in elements.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Eight {
  T e[8];
};
// The power of two that takes the largest weight to [2^14, 2^15).
struct ScaleArgs {
  const float *weights;
  const int32_t *targets;
  int64_t n, m;
  float *scale;  // nullable: not wanted
};
__device__ __forceinline__ void find_scale(const ScaleArgs &a) {
  __shared__ float tops[4];
  float top = 0.0f;
  for (int64_t r = threadIdx.x; r < a.n; r += 256) {
    const int32_t t = a.targets[r];
    const float w = a.weights ? fabsf(a.weights[r]) : 1.0f;
    if (t >= 0 && t < a.m && w < __builtin_inff()) top = fmaxf(top, w);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) *a.scale = scale_for(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
}

// One launch for both sides and the scale: `blocks` of each side, and one.
struct LayBoth {
  LayArgs side[2];
  uint32_t blocks[2];
  ScaleArgs scale;
};
template <typename T>
__global__ __launch_bounds__(256) void lay_kernel(LayBoth both) {
  constexpr int NP = kPlanes<T>;
  __shared__ __attribute__((aligned(16))) uint16_t tile[NP][64][72];
  uint32_t id = blockIdx.x;
  if (id >= both.blocks[0] + both.blocks[1]) {
    find_scale(both.scale);
    return;
  }
  const bool second = id >= both.blocks[0];
  if (second) id -= both.blocks[0];
  const LayArgs a = second ? both.side[1] : both.side[0];
  float whole = 1.0f;
  if constexpr (NP > 1)
    if (a.turned) whole = turned_scale(a.tops);
  const uint32_t across = (uint32_t)((a.cols + 63) / 64);
  const int64_t r0 = (int64_t)(id / across) * 64, c0 = (int64_t)(id % across) * 64;
  const int in = (threadIdx.x & 7) * 8;
  const T *const x = static_cast<const T *>(a.x);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = (threadIdx.x >> 3) + 32 * h;
    const int64_t r = r0 + i, c = c0 + in;
    Eight<T> t{};
    bool out = true;
    if (r < a.rows) {
      if (c + 8 <= a.cols) t = *reinterpret_cast<const Eight<T> *>(x + r * a.ld + c);
      else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < a.cols) t.e[e] = x[r * a.ld + c + e];
      }
      out = a.turned && a.mask.out(r);
    }
    const auto planes = [&](float scale, u32x4 (&w)[NP]) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        uint16_t lo[NP], hi[NP];
        split(scaled(t.e[e], scale), lo);
        split(scaled(t.e[e + 1], scale), hi);
#pragma unroll
        for (int p = 0; p < NP; ++p) w[p][e / 2] = (uint32_t)lo[p] | (uint32_t)hi[p] << 16;
      }
    };
    u32x4 w[NP];
    if (a.packed && r < a.rows && c < a.ld_p) {
      planes(NP > 1 ? a.row_scale[r] : 1.0f, w);
#pragma unroll
      for (int p = 0; p < NP; ++p)
        *reinterpret_cast<u32x4 *>(a.packed + p * a.plane_p + r * a.ld_p + c) = w[p];
    }
    if (!a.turned) continue;
    planes(whole, w);
#pragma unroll
    for (int p = 0; p < NP; ++p) *reinterpret_cast<u32x4 *>(&tile[p][i][in]) = out ? u32x4{} : w[p];
  }
  if (!a.turned) return;
  __syncthreads();
  // a thread takes 8 rows of one column: neighbouring threads neighbouring columns
  const int c_in = threadIdx.x & 63;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r_in = ((threadIdx.x >> 6) + 4 * h) * 8;
    const int64_t c = c0 + c_in, r = r0 + r_in;
    if (c >= a.cols || r >= a.ld_t) continue;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = (uint32_t)tile[p][r_in + 2 * e][c_in] | (uint32_t)tile[p][r_in + 2 * e + 1][c_in] << 16;
      *reinterpret_cast<u32x4 *>(a.turned + p * a.plane_t + c * a.ld_t + r) = w;
    }
  }
}

// ---------------------------------------------------------------------------
// 1. logits

// How e^(z - max) is kept, in units of 2^-kShift, so that small ones stay
// normal numbers.
// bf16: as fp16 (an error of 2^-11 where G is rounded by 2^-8).
struct CodeBf16 {
  using Word = uint16_t;
  static constexpr int kShift = 15;
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  }
  static __device__ __forceinline__ float value(uint32_t w) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)w);
  }
};
// fp16: as fp16 whose sign's bit is one more of mantissa, which is float32's own
// bits of p 2^-96 but the last 12: 5 bits of exponent, 11 of mantissa (an error
// of 2^-12 where G is rounded by 2^-11), running out gradually below 2^-30. (4
// bits of exponent and 12 of mantissa ran out below 2^-14, so that items beside
// one that is nearly certain lost their gradients.)
struct CodeF16 {
  using Word = uint16_t;
  static constexpr int kShift = 0;
  static __device__ __forceinline__ uint32_t one(float p) {
    return (__builtin_bit_cast(uint32_t, p * 0x1p-96f) + 0x800u) >> 12;
  }
  static __device__ __forceinline__ uint32_t two(float a, float b) { return one(a) | one(b) << 16; }
  static __device__ __forceinline__ float value(uint32_t w) {
    return __builtin_bit_cast(float, w << 12) * 0x1p96f;
  }
};
struct CodeF32 {
  using Word = float;
  static constexpr int kShift = 0;
};

struct LogitArgs {
  GemmArgs g;         // q: the piece's queries, p: items
  // Logits stand as the sums themselves, or with a bias as f (1 / tau in two parts; else 1) times the
  // sums and the bias as it is: scaled, one of the type's lowest value would be -inf. c (log2(e) / tau,
  // or with a bias log2(e)) takes their differences to powers of two.
  float c, f, f_low;
  const float *bias;  // nullable
  const float *scale_q, *scale_p;  // float32: those of the packed rows
  const int32_t *targets;
  void *code;  // nullable: uint16 (float32: float) [rows][ld]
  int64_t ld;
  float2 *stats;  // [rows][blocks]: of a block of columns (max of z, sum of 2^(c (z - max)))
  int64_t blocks;
  float *z_target;
};

constexpr double kLog2e = 1.44269504088896340736;

template <class Op, class Code, int TC, int TR, int WC, int WR>
__global__ __launch_bounds__(64 * WC * WR) void ce_logits_kernel(LogitArgs a) {
  using Tile = GemmTile<Op, TC, TR, WC, WR>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tile::kLds];
  Tile t(a.g, lds);
  using Word = typename Code::Word;
  constexpr float kInf = __builtin_inff();
  constexpr int FC = Tile::kFragC, FR = Tile::kFragR;
  const int64_t rows = a.g.q.rows, cols = a.g.p.rows;
  const int wave_col = t.wc * (TC / WC);
  // float32: the factor's second part, so that its rounding does not change the temperature
  constexpr bool kLow = sizeof(Word) == 4;
  int32_t target[FR];
  int up[FR];  // float32: exponents of the rows' scales
  const auto take = [&] {
#pragma unroll
    for (int j = 0; j < FR; ++j) {
      const int64_t r = t.at.row0 + t.row_of(j);
      target[j] = a.targets[r < rows ? r : rows - 1];
      if (kLow) up[j] = exponent_of(a.scale_q[r < rows ? r : rows - 1]);
    }
    if constexpr (kLow) {
      float s[FC][4];
      t.of_columns(a.scale_p, 1.0f, s);
#pragma unroll
      for (int i = 0; i < FC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int up_c = exponent_of(s[i][e]);
#pragma unroll
          for (int j = 0; j < FR; ++j)
            t.acc[i][j][e] = __builtin_amdgcn_ldexpf(t.acc[i][j][e], -(up_c + up[j]));
        }
    }
    if (!a.bias && t.at.col0 + TC <= cols) return;
    float b[FC][4];
    if (a.bias) {
      t.of_columns(a.bias, -kInf, b);
    } else {
#pragma unroll
      for (int i = 0; i < FC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) b[i][e] = t.at.col0 + t.col_of(i) + e < cols ? 0.0f : -kInf;
    }
#pragma unroll
    for (int i = 0; i < FC; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < FR; ++j) {  // a column that is struck out has no logit, whatever its item holds
          const float y = kLow && a.f_low != 0.0f ? __builtin_fmaf(t.acc[i][j][e], a.f_low, b[i][e]) : b[i][e];
          t.acc[i][j][e] = b[i][e] == -kInf ? -kInf : __builtin_fmaf(t.acc[i][j][e], a.f, y);
        }
  };
  const auto put_all = [&](auto whole) {
    const int64_t block = (t.at.col0 + wave_col) / (TC / WC);
#pragma unroll
    for (int j = 0; j < FR; ++j) {
      const int64_t r = t.at.row0 + t.row_of(j);
      float top = -kInf;
#pragma unroll
      for (int i = 0; i < FC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, t.acc[i][j][e]);
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      // the target's logit, where it is one of this wave's columns
      const int first = (int)(target[j] - t.at.col0);
      if (r < rows && (uint32_t)(first - wave_col) < (uint32_t)(TC / WC)) {
#pragma unroll
        for (int i = 0; i < FC; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (first == t.col_of(i) + e) a.z_target[r] = t.acc[i][j][e];
      }
      const float base = top == -kInf ? 0.0f : top;
      float sum = 0.0f;
      typename QuadOf<Word>::Bits w[FC];
#pragma unroll
      for (int i = 0; i < FC; ++i) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // The difference to the largest first: 0 there, and exact near by, however large both are. Then
          // the shift. (A second part of c would be a part of this rounding.)
          p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(t.acc[i][j][e] - base, a.c, (float)Code::kShift));
          sum += p[e];
        }
        if constexpr (sizeof(Word) == 2) w[i] = {Code::two(p[0], p[1]), Code::two(p[2], p[3])};
        else w[i] = quad_of<float>(p);
      }
      if (a.code)  // rows of codes are padded to a multiple of 64
        t.template store<Word, whole.value, true>(j, w, static_cast<Word *>(a.code), a.ld, rows,
                                            (cols + 63) & ~63ll);
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      if (r < rows && t.lane < 16 && t.at.col0 + wave_col < cols)
        a.stats[r * a.blocks + block] = {top, sum * (1.0f / (float)(1 << Code::kShift))};
    }
  };
  const auto put = [&] {
    const bool whole = t.full();
    if (whole) put_all(std::true_type{});
    else put_all(std::false_type{});
    return a.code && whole;
  };
  gemm_tiles<Tile::template kStores<Word>>(t, a.g, Op{}, blockIdx.x, [&] { t.clear(); }, take, put);
}

// ---------------------------------------------------------------------------
// 2. sums, and the gradient of the logits

struct GradArgs {
  const float2 *stats;
  int64_t rows, cols;
  int32_t blocks, block;  // their number and columns
  const float *z_target;
  double unit;  // a difference of logits times unit is one of powers of two
  const float *weights;  // nullable
  const int32_t *targets;
  const float *scale;  // nullable: 1
  float *loss;
  const void *code;  // [rows][ld]
  int64_t ld;
  uint16_t *g;  // planes of [rows][ld]; a 16-bit code's own place
  int64_t plane_g;
  float *factor;  // [rows]: 0 where a row has no gradient
};

// Sums beyond a block in float64, as are differences of maxima, whose size does not matter so.
struct Running {
  float top;
  double sum;
  __device__ __forceinline__ void join(float t, double s, double unit) {
    const float m = fmaxf(top, t);
    if (m == -__builtin_inff()) sum += s;  // 0, or NaN
    else
      sum = sum * (double)__builtin_amdgcn_exp2f((float)(((double)top - (double)m) * unit)) +
            s * (double)__builtin_amdgcn_exp2f((float)(((double)t - (double)m) * unit));
    top = m;
  }
};
template <int LANES>
__device__ __forceinline__ Running run_row(const float2 *stats, int32_t blocks, int lane, int step,
                                           double unit) {
  Running x{-__builtin_inff(), 0.0};
  for (int32_t b = lane; b < blocks; b += step) {
    const float2 s = stats[b];
    x.join(s.x, (double)s.y, unit);
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    const float t = __shfl_xor(x.top, o, 64);
    const double s = __shfl_xor(x.sum, o, 64);
    x.join(t, s, unit);
  }
  return x;
}
// The loss of a row, and whether it has one: its target is a column and some
// column is left (its largest logit adds 1 to the sum, or NaN).
__device__ __forceinline__ bool loss_of(const GradArgs &a, int64_t r, const Running &x, double *loss) {
  const int32_t t = a.targets[r];
  if (t < 0 || t >= a.cols || x.sum == 0.0) {
    *loss = 0.0;
    return false;
  }
  *loss = (((double)x.top - (double)a.z_target[r]) * a.unit + log2(x.sum)) * 0.69314718055994530942;
  return true;
}

// Losses alone: 16 lanes a row.
__global__ __launch_bounds__(256) void ce_loss_kernel(GradArgs a) {
  const int64_t r = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int lane = threadIdx.x & 15;
  const Running x = run_row<16>(a.stats + (r < a.rows ? r : 0) * a.blocks, a.blocks, lane, 16, a.unit);
  if (r >= a.rows || lane != 0) return;
  double loss;
  loss_of(a, r, x, &loss);
  a.loss[r] = (float)loss;
}

// A workgroup a row, 8 values a thread and step; the first ones are on their
// way while the row's sums are joined (the first four: 1001 x 100,000 fp16 391
// instead of 385 us of all, others the same). Bound by memory: codes read, G
// written in their place.
template <typename T, class Code>
__global__ __launch_bounds__(256) void ce_grad_kernel(GradArgs a) {
  constexpr int NP = kPlanes<T>;
  __shared__ Running parts[4];
  const int64_t r = blockIdx.x;
  const int64_t vecs = (a.cols + 63) / 64 * 8;  // G is filled with zeros to whole steps of a product
  using Word = typename Code::Word;
  struct Codes {
    u32x4 w[sizeof(Word) / 2];
  };
  const Word *const code = static_cast<const Word *>(a.code) + r * a.ld;
  const auto fetch = [&](int64_t v) { return *reinterpret_cast<const Codes *>(code + v * 8); };
  Codes ahead = {};
  if (threadIdx.x < vecs) ahead = fetch(threadIdx.x);

  const float2 *const stats = a.stats + r * a.blocks;
  const Running mine = run_row<64>(stats, a.blocks, threadIdx.x, 256, a.unit);
  if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = mine;
  __syncthreads();
  Running x = parts[0];
  for (int i = 1; i < 4; ++i) x.join(parts[i].top, parts[i].sum, a.unit);
  double loss;
  const bool takes = loss_of(a, r, x, &loss);
  const float factor =
      takes ? (a.weights ? a.weights[r] : 1.0f) * (a.scale ? *a.scale : 1.0f) : 0.0f;
  if (threadIdx.x == 0) {
    a.loss[r] = (float)loss;
    a.factor[r] = factor;
  }
  const double top = (double)x.top, rest = log2(x.sum) + (double)Code::kShift;
  const float at_target = takes ? (float)expm1(-loss) * factor : 0.0f;
  const int32_t target = a.targets[r];

  const auto put = [&](int64_t v, const Codes &c) {
    const int64_t col = v * 8;
    uint16_t o[NP][8] = {};
    if (factor != 0.0f) {
      const float f = col < a.cols
                          ? __builtin_amdgcn_exp2f(
                                (float)(((double)stats[col / a.block].x - top) * a.unit - rest)) *
                                factor
                          : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float p;
        if constexpr (sizeof(Word) == 2) {
          p = Code::value((c.w[0][e / 2] >> (16 * (e & 1))) & 0xffffu);
        } else {
          const uint32_t u = c.w[e / 4][e & 3];
          p = __builtin_bit_cast(float, u);
        }
        const float g = col + e < a.cols ? (col + e == target ? at_target : p * f) : 0.0f;
        uint16_t w[NP];
        if constexpr (NP == 1) w[0] = from_f32<T>(g).u;
        else split(g, w);
#pragma unroll
        for (int k = 0; k < NP; ++k) o[k][e] = w[k];
      }
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = (uint32_t)o[k][2 * e] | (uint32_t)o[k][2 * e + 1] << 16;
      *reinterpret_cast<u32x4 *>(a.g + k * a.plane_g + r * a.ld + col) = w;
    }
  };
  if (threadIdx.x < vecs) put(threadIdx.x, ahead);
  for (int64_t v = threadIdx.x + 256; v < vecs; v += 256) put(v, fetch(v));
}

// ---------------------------------------------------------------------------
// 3. products with the gradient

// Which rows of the gradient are zeros whatever the sums say.
struct OutMask {
  const float *factor;  // nullable: rows without one
  const float *bias;   // nullable: items struck out
  __device__ __forceinline__ bool out(int64_t r) const {
    return (factor && factor[r] == 0.0f) || (bias && bias[r] == -__builtin_inff());
  }
};

struct ProductArgs {
  GemmArgs g;
  const float *before;  // nullable: [rows][cols] sums of earlier pieces
  float *part;          // sums of the tail's parts: part z, from the tail's first row, at z * stride
  int64_t stride, tail_row;
  void *out;
  int64_t ld;
  int32_t dtype;
  float alpha;
  const float *scale;  // nullable: G's, which is divided out
  const float *tops;   // float32: the maxima behind the turned operand's scale, likewise
  OutMask mask;
};
// The exponent of both scales.
__device__ __forceinline__ int ups_of(const float *scale, const float *tops) {
  int up = scale ? exponent_of(*scale) : 0;
  if (tops) {
    float top = 0.0f;
    for (int i = threadIdx.x & 63; i < kMaxBlocks; i += 64) top = fmaxf(top, tops[i]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    up += exponent_of(scale_for(top));
  }
  return up;
}

__device__ __forceinline__ void put_typed(void *out, int32_t dtype, int64_t at, int64_t col,
                                          int64_t cols, const float v[4]) {
  if (dtype == SPS_F32) put_four<float>(static_cast<float *>(out) + at, col, cols, v);
  else if (dtype == SPS_F16) put_four<f16_t>(static_cast<f16_t *>(out) + at, col, cols, v);
  else put_four<bf16_t>(static_cast<bf16_t *>(out) + at, col, cols, v);
}

// The tile's sums times alpha 2^-up, to rows of T.
template <typename T, bool FULL, class Tile>
__device__ __forceinline__ void product_out(Tile &t, T *out, int64_t ld, float alpha, int up,
                                            const OutMask &mask) {
  const int64_t rows = t.a.q.rows, cols = t.a.p.rows;
#pragma unroll
  for (int j = 0; j < Tile::kFragR; ++j) {
    const int64_t r = t.at.row0 + t.row_of(j);
    const bool zero = r < rows && mask.out(r);
    typename QuadOf<T>::Bits w[Tile::kFragC];
#pragma unroll
    for (int i = 0; i < Tile::kFragC; ++i) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = zero ? 0.0f : __builtin_amdgcn_ldexpf(t.acc[i][j][e] * alpha, -up);
      w[i] = quad_of<T>(v);
    }
    t.template store<T, FULL, false>(j, w, out, ld, rows, cols);
  }
}

template <class Op, bool QT, int TC, int TR, int WC, int WR>
__device__ __forceinline__ void product_tiles(const ProductArgs &a, uint32_t first, uint8_t *lds) {
  using Tile = GemmTile<Op, TC, TR, WC, WR, QT>;
  Tile t(a.g, lds);
  const int up = ups_of(a.scale, a.tops);
  using Type = typename Op::Type;  // the rows' own: that of the products
  const auto start = [&] {
    if (a.before && t.at.z < 0) t.start(a.before, a.g.q.rows, a.g.p.rows);
    else t.clear();
  };
  const auto put_all = [&](auto whole) {
    constexpr bool FULL = whole.value;
    if (t.at.z >= 0)
      product_out<float, FULL>(t, a.part + t.at.z * a.stride - a.tail_row * a.g.p.rows, a.g.p.rows,
                               1.0f, 0, {});
    else if (a.dtype == SPS_F32)
      product_out<float, FULL>(t, static_cast<float *>(a.out), a.ld, a.alpha, up, a.mask);
    else product_out<Type, FULL>(t, static_cast<Type *>(a.out), a.ld, a.alpha, up, a.mask);
  };
  const auto put = [&] {
    const bool whole = t.full();
    if (whole) put_all(std::true_type{});
    else put_all(std::false_type{});
    return whole;
  };
  // the fewest stores of the three
  gemm_tiles<Tile::template kStores<Type>>(t, a.g, Op{}, first, start, [] {}, put);
}

// Both products in one launch, either without tiles where it is not wanted:
// the items' tiles go on where the queries' end, so that no part of the card
// waits for the last of these.
struct ProductsArgs {
  ProductArgs queries, items;
};
template <class Op, int TC, int TR, int WC, int WR>
__global__ __launch_bounds__(64 * WC * WR) void ce_products_kernel(ProductsArgs a) {
  constexpr int kLds = GemmTile<Op, TC, TR, WC, WR, false>::kLds;
  static_assert((kLds == GemmTile<Op, TC, TR, WC, WR, true>::kLds), "one size");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  product_tiles<Op, false, TC, TR, WC, WR>(a.queries, blockIdx.x, lds);
  const uint32_t before = gemm_all(a.queries.g) % gridDim.x;
  product_tiles<Op, true, TC, TR, WC, WR>(a.items, (blockIdx.x + gridDim.x - before) % gridDim.x, lds);
}

struct JoinArgs {
  const float *part;
  const float *before;  // nullable: [first + rows][cols]
  int64_t stride, first, rows, cols;
  int32_t splits;
  void *out;
  int64_t ld;
  int32_t dtype;
  float alpha;
  const float *scale, *tops;
  OutMask mask;
};
// Of both products: `blocks` workgroups each.
struct JoinBoth {
  JoinArgs side[2];
  uint32_t blocks[2];
};

// The splits' sums in their order, four values a thread.
__global__ __launch_bounds__(256) void ce_join_kernel(JoinBoth both) {
  const bool second = blockIdx.x >= both.blocks[0];
  const JoinArgs a = second ? both.side[1] : both.side[0];
  const uint32_t block = second ? blockIdx.x - both.blocks[0] : blockIdx.x;
  const uint32_t blocks = second ? both.blocks[1] : both.blocks[0];
  const int64_t per = (a.cols + 3) / 4, all = a.rows * per;
  const int up = ups_of(a.scale, a.tops);
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < all; i += (int64_t)blocks * 256) {
    const int64_t r = i / per, c = (i - r * per) * 4;
    float v[4] = {};
    if (a.before)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.cols) v[e] = a.before[(a.first + r) * a.cols + c + e];
    for (int32_t z = 0; z < a.splits; ++z) {
      const float *const p = a.part + z * a.stride + r * a.cols + c;
      if (c + 4 <= a.cols) {
        const Four<float> f = *reinterpret_cast<const Four<float> *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += f.e[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < a.cols) v[e] += p[e];
      }
    }
    const bool zero = a.mask.out(a.first + r);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = zero ? 0.0f : __builtin_amdgcn_ldexpf(v[e] * a.alpha, -up);
    put_typed(a.out, a.dtype, (a.first + r) * a.ld, c, a.cols, v);
  }
}

__global__ __launch_bounds__(256) void zero_rows_kernel(uint8_t *out, int64_t rows, int64_t bytes,
                                                        int64_t stride) {
  const int64_t words = bytes / 2, all = rows * words;  // 16-bit elements at the least
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256)
    *reinterpret_cast<uint16_t *>(out + (i / words) * stride + (i % words) * 2) = 0;
}

}  // namespace sps

using sps::ceil_div;
using sps::GemmOperand;
using sps::set_error;

namespace {

// 256 rows of G, or of a transposed operand, stay below 2^31 bytes.
constexpr int64_t kMaxRows = 4000000;
constexpr int64_t kMaxDim = 1ll << 16;
// Bytes of a piece's codes and gradients, and of statistics where there are no
// codes. Large pieces, since the items' sums go on from piece to piece and each
// ends with workgroups that wait: 8192 x 100,000 x 1024 bf16 5050 us in one piece
// (1.6 GB), 5230 in two, 6370 in pieces of 256 MB.
constexpr int64_t kPieceBytes = 1ll << 31;
constexpr int64_t kStatBytes = 1ll << 28;
constexpr int64_t kMaxPiece = 1ll << 20;

int64_t up(int64_t x, int64_t to) { return ceil_div(x, to) * to; }

struct Shape {
  int64_t n, m, d;
  int32_t dtype;
  bool gq, gi;  // which gradients
  bool pack_q, pack_i;
  int64_t piece;     // rows of a piece, a multiple of 64
  int64_t at_once;   // of them there are
  int64_t ld_g;      // items, padded
  int32_t block;     // columns of a block of statistics
  int64_t blocks;
  sps::TilePlan plan_l;  // of the logits
};

int64_t steps_of(const Shape &s, int64_t k) {
  return ceil_div(k * 2, sps::kStep) * (s.dtype == SPS_F32 ? sps::kSegments : 1);
}
constexpr int kMostSplits = 64;
// The plans of both products, which are one launch: tiles of one size, that
// of the lesser time together.
struct PlanBoth {
  bool big;
  sps::TilePlan q, i;
};
PlanBoth plan_products(const Shape &s, int64_t rows) {
  PlanBoth best{};
  double least = 1e300;
  for (const bool big : {false, true}) {
    PlanBoth p{big, {}, {}};
    if (s.gq) p.q = sps::plan_tiles(big, rows, s.d, steps_of(s, s.m), kMostSplits);
    if (s.gi) p.i = sps::plan_tiles(big, s.m, s.d, steps_of(s, rows), kMostSplits);
    if (p.q.us + p.i.us < least) {
      least = p.q.us + p.i.us;
      best = p;
    }
  }
  return best;
}
int64_t part_values(const sps::TilePlan &p, int64_t rows, int64_t cols) {
  return p.tail_r ? p.splits * (rows - p.tail_row()) * cols : 0;
}

struct Layout {
  size_t scale, tops_q, tops_i, rows_q, rows_i, factor, z_target, stats, packed_q, packed_i, turned_q, turned_i, code, g, part_q, part_i,
      sum_i, total;
};

int planes(const Shape &s) { return s.dtype == SPS_F32 ? 2 : 1; }

// Rows of 16-bit values that hold `k`, in whole 128 bytes. (Rows of a large power of two, and steps
// begun elsewhere in every column of tiles: 4096 x 32,768 x 1024 849 against 847 us, 4000 x 20,000 x
// 4096 in 8 bits 291 against 292.)
int64_t turned_ld(int64_t rows) { return up(rows, 64); }
int64_t packed_ld(const Shape &s) { return up(s.d, 8); }

// 16-byte rows and whole 16-byte chunks of k are read where they lie
bool must_pack(const sps_scores *x) {
  return x->dtype == SPS_F32 || x->n_cols % 8 || (x->ld * 2) % 16 ||
         reinterpret_cast<uintptr_t>(x->data) % 16;
}

Shape shape_of(const sps_scores *q, const sps_scores *i, bool gq, bool gi) {
  Shape s{};
  s.n = q->n_rows;
  s.m = i->n_rows;
  s.d = q->n_cols;
  s.dtype = q->dtype;
  s.gq = gq;
  s.gi = gi;
  s.pack_q = must_pack(q);
  s.pack_i = must_pack(i);
  s.ld_g = turned_ld(s.m);
  const bool grad = gq || gi;
  const int64_t each = s.dtype == SPS_F32 ? 8 : 2;
  s.block = 64;
  int64_t rows = grad ? kPieceBytes / (s.ld_g * each) : kStatBytes / (8 * ceil_div(s.m, 64));
  rows = rows / 256 * 256;
  if (rows < 256) rows = 256;
  if (rows > kMaxPiece) rows = kMaxPiece;
  s.piece = rows < s.n ? up(ceil_div(s.n, ceil_div(s.n, rows)), 256) : up(s.n, 64);
  s.at_once = s.piece < s.n ? s.piece : s.n;
  s.plan_l = sps::plan_tiles(s.at_once, s.m, steps_of(s, s.d), 1);
  s.block = s.plan_l.big ? 128 : 64;
  s.blocks = ceil_div(s.m, s.block);
  return s;
}

Layout layout_of(const Shape &s) {
  Layout L{};
  size_t at = 0;
  const auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += (size_t)up(bytes, 256);
    return here;
  };
  const int p = planes(s);
  L.scale = take(4);
  if (p > 1) {
    L.tops_q = take(sps::kMaxBlocks * 4);
    L.tops_i = take(sps::kMaxBlocks * 4);
    L.rows_q = take(s.n * 4);
    L.rows_i = take(s.m * 4);
  }
  L.z_target = take(s.piece * 4);
  L.stats = take(s.blocks * s.piece * 8);
  if (s.pack_q) L.packed_q = take(s.n * packed_ld(s) * 2 * p);
  if (s.pack_i) L.packed_i = take(s.m * packed_ld(s) * 2 * p);
  if (s.gq || s.gi) {
    L.factor = take(s.piece * 4);
    L.code = take(s.piece * s.ld_g * (p > 1 ? 4 : 2));
    L.g = p > 1 ? take(s.piece * s.ld_g * 2 * p) : L.code;
    if (s.gq) {
      L.turned_i = take(s.d * turned_ld(s.m) * 2 * p);
    }
    if (s.gi) {
      L.turned_q = take(s.d * turned_ld(s.n) * 2 * p);
      if (s.piece < s.n) L.sum_i = take(s.m * s.d * 4);
    }
    // parts of the products, also of a last piece that is shorter
    int64_t pq = 0, pi = 0;
    const auto count = [&](int64_t rows) {
      const PlanBoth p = plan_products(s, rows);
      const int64_t q = part_values(p.q, rows, s.d), i = part_values(p.i, s.m, s.d);
      pq = pq > q ? pq : q;
      pi = pi > i ? pi : i;
    };
    count(s.at_once);
    if (s.n % s.piece && s.n > s.piece) count(s.n % s.piece);
    L.part_q = take(pq * 4);
    L.part_i = take(pi * 4);
  }
  L.total = at;
  return L;
}

sps_status check_shape(const sps_scores *q, const sps_scores *i, const char *what) {
  sps_status st = sps::check_scores(q, what);
  if (st == SPS_OK) st = sps::check_scores(i, what);
  if (st != SPS_OK) return st;
  if (q->dtype != i->dtype)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: queries and items of different types", what);
  if (q->n_cols != i->n_cols)
    return set_error(SPS_ERR_DIM_MISMATCH, "%s: queries have %lld dims, items %lld", what,
                     (long long)q->n_cols, (long long)i->n_cols);
  if (q->n_cols < 1) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: no dims", what);
  if (q->n_cols > kMaxDim)
    return set_error(SPS_ERR_UNSUPPORTED, "%s: at most %lld dims", what, (long long)kMaxDim);
  if (q->n_rows > kMaxRows || i->n_rows > kMaxRows)
    return set_error(SPS_ERR_UNSUPPORTED, "%s: at most %lld queries and items", what,
                     (long long)kMaxRows);
  const int64_t most = sps::kMostBytes / 256 / 4;  // a tile's rows in 31 bits of bytes
  if (q->ld > most || i->ld > most)
    return set_error(SPS_ERR_OVERFLOW, "%s: ld must be at most %lld", what, (long long)most);
  // the tiles of both sides that are laid out, and one workgroup
  return sps::check_grid((ceil_div(q->n_rows, 64) + ceil_div(i->n_rows, 64)) * ceil_div(q->n_cols, 64) + 1,
                         256, what);
}

sps_status check_out(const sps_scores *q, const sps_scores *i, const sps_scores *of,
                     const void *grad, int32_t dtype, int64_t ld, const char *what) {
  if (!grad) return SPS_OK;
  const sps_scores view{grad, dtype, of->n_rows, of->n_cols, ld, 0};
  const sps_status st = sps::check_scores(&view, what);
  if (st != SPS_OK) return st;
  if (dtype != q->dtype && dtype != SPS_F32)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: the gradient's type is the rows' or float32",
                     what);
  const int64_t sg = sps::dtype_size(dtype), sx = sps::dtype_size(q->dtype);
  const sps::RowBytes g{grad, of->n_rows, of->n_cols * sg, ld * sg};
  if (sps::rows_overlap(g, {q->data, q->n_rows, q->n_cols * sx, q->ld * sx}) ||
      sps::rows_overlap(g, {i->data, i->n_rows, i->n_cols * sx, i->ld * sx}))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: a gradient overlaps the rows", what);
  return SPS_OK;
}

void launch_lay(int32_t dtype, sps::LayBoth *a, hipStream_t s) {
  for (int i = 0; i < 2; ++i) {
    const sps::LayArgs &x = a->side[i];
    a->blocks[i] = x.packed || x.turned ? (uint32_t)(ceil_div(x.rows, 64) * ceil_div(x.cols, 64)) : 0;
  }
  const dim3 grid(a->blocks[0] + a->blocks[1] + (a->scale.scale ? 1 : 0)), block(256);
  if (grid.x == 0) return;
  if (dtype == SPS_F32) hipLaunchKernelGGL((sps::lay_kernel<float>), grid, block, 0, s, *a);
  else if (dtype == SPS_F16) hipLaunchKernelGGL((sps::lay_kernel<sps::f16_t>), grid, block, 0, s, *a);
  else hipLaunchKernelGGL((sps::lay_kernel<sps::bf16_t>), grid, block, 0, s, *a);
}

template <class Op, class Code>
void launch_logits(const sps::TilePlan &plan, sps::LogitArgs a, hipStream_t s) {
  plan.give(&a.g);
  const dim3 grid(plan.grid());
  if (plan.big) hipLaunchKernelGGL((sps::ce_logits_kernel<Op, Code, 256, 256, 2, 4>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((sps::ce_logits_kernel<Op, Code, 128, 128, 2, 2>), grid, dim3(256), 0, s, a);
}

template <class Op>
void launch_product_tiles(bool big, uint32_t grid, const sps::ProductsArgs &a, hipStream_t s) {
  if (big) hipLaunchKernelGGL((sps::ce_products_kernel<Op, 256, 256, 2, 4>), dim3(grid), dim3(512), 0, s, a);
  else hipLaunchKernelGGL((sps::ce_products_kernel<Op, 128, 128, 2, 2>), dim3(grid), dim3(256), 0, s, a);
}

// The products and, where a tail was split, the sums of its parts.
void launch_products(int32_t dtype, const PlanBoth &plan, sps::ProductsArgs *a, hipStream_t s) {
  sps::JoinBoth join{};
  const sps::TilePlan *const plans[2] = {&plan.q, &plan.i};
  sps::ProductArgs *const sides[2] = {&a->queries, &a->items};
  for (int k = 0; k < 2; ++k) {
    const sps::TilePlan &p = *plans[k];
    sps::ProductArgs &x = *sides[k];
    p.give(&x.g);
    if (p.tail_r == 0) continue;
    x.tail_row = p.tail_row();
    const int64_t rows = x.g.q.rows - x.tail_row, cols = x.g.p.rows;
    x.stride = rows * cols;
    join.side[k] = {x.part, x.before, x.stride, x.tail_row, rows,    cols,  p.splits,
                    x.out,  x.ld,     x.dtype,  x.alpha,    x.scale, x.tops, x.mask};
    const int64_t blocks = ceil_div(rows * ceil_div(cols, 4), 256);
    join.blocks[k] = (uint32_t)(blocks < 4096 ? blocks : 4096);
  }
  const int64_t all = plan.q.all() + plan.i.all(), at_once = plan.big ? sps::kCus : 2 * sps::kCus;
  const uint32_t grid = (uint32_t)(all < at_once ? all : at_once);
  if (dtype == SPS_F32) launch_product_tiles<sps::OpF32>(plan.big, grid, *a, s);
  else if (dtype == SPS_F16) launch_product_tiles<sps::OpF16>(plan.big, grid, *a, s);
  else launch_product_tiles<sps::OpBf16>(plan.big, grid, *a, s);
  if (join.blocks[0] + join.blocks[1])
    hipLaunchKernelGGL(sps::ce_join_kernel, dim3(join.blocks[0] + join.blocks[1]), dim3(256), 0, s, join);
}

void launch_grad(int32_t dtype, const sps::GradArgs &a, hipStream_t s) {
  const dim3 grid((uint32_t)a.rows), block(256);
  if (dtype == SPS_F32)
    hipLaunchKernelGGL((sps::ce_grad_kernel<float, sps::CodeF32>), grid, block, 0, s, a);
  else if (dtype == SPS_F16)
    hipLaunchKernelGGL((sps::ce_grad_kernel<sps::f16_t, sps::CodeF16>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((sps::ce_grad_kernel<sps::bf16_t, sps::CodeBf16>), grid, block, 0, s, a);
}

void launch_zero(void *out, int64_t rows, int64_t bytes, int64_t stride, hipStream_t s) {
  if (rows == 0 || bytes == 0) return;
  int64_t blocks = ceil_div(rows * (bytes / 2), 256);
  if (blocks > 4096) blocks = 4096;
  hipLaunchKernelGGL(sps::zero_rows_kernel, dim3((uint32_t)blocks), dim3(256), 0, s,
                     static_cast<uint8_t *>(out), rows, bytes, stride);
}

}  // namespace

extern "C" {

sps_status sps_dense_ce_workspace_size(const sps_scores *queries, const sps_scores *items,
                                       int32_t grad_queries, int32_t grad_items, size_t *bytes) {
  const char *what = "sps_dense_ce_workspace_size";
  if (!bytes) return set_error(SPS_ERR_INVALID_ARGUMENT, "NULL output pointer");
  const sps_status st = check_shape(queries, items, what);
  if (st != SPS_OK) return st;
  *bytes = queries->n_rows && items->n_rows
               ? layout_of(shape_of(queries, items, grad_queries != 0, grad_items != 0)).total
               : 0;
  return SPS_OK;
}

sps_status sps_dense_ce(const sps_scores *queries, const sps_scores *items, const int32_t *targets,
                        const float *bias, float temperature, const float *row_weights, float *loss,
                        void *grad_queries, int64_t ld_queries, void *grad_items, int64_t ld_items,
                        int32_t grad_dtype, void *workspace, size_t workspace_bytes, void *stream) {
  const char *what = "sps_dense_ce";
  sps_status st = check_shape(queries, items, what);
  if (st == SPS_OK)
    st = check_out(queries, items, queries, grad_queries, grad_dtype, ld_queries, what);
  if (st == SPS_OK) st = check_out(queries, items, items, grad_items, grad_dtype, ld_items, what);
  if (st != SPS_OK) return st;
  const int64_t n = queries->n_rows, m = items->n_rows, d = queries->n_cols;
  const int64_t sg = sps::dtype_size(grad_dtype);
  if (grad_queries && grad_items &&
      sps::rows_overlap({grad_queries, n, d * sg, ld_queries * sg}, {grad_items, m, d * sg, ld_items * sg}))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: the gradients overlap", what);
  // what is written is so while the rest is still read, by a later piece of the rows at the latest
  const int64_t sx = sps::dtype_size(queries->dtype);
  const auto some = [](const void *at, sps::RowBytes b) { return at ? b : sps::RowBytes{}; };
  const sps::RowBytes losses = some(loss, {loss, 1, n * 4, n * 4});
  const sps::RowBytes grads[2] = {some(grad_queries, {grad_queries, n, d * sg, ld_queries * sg}),
                                  some(grad_items, {grad_items, m, d * sg, ld_items * sg})};
  const sps::RowBytes rows[2] = {{queries->data, n, d * sx, queries->ld * sx},
                                 {items->data, m, d * sx, items->ld * sx}};
  const sps::RowBytes lists[3] = {some(targets, {targets, 1, n * 4, n * 4}),
                                  some(bias, {bias, 1, m * 4, m * 4}),
                                  some(row_weights, {row_weights, 1, n * 4, n * 4})};
  const auto in_any = [](const sps::RowBytes &x, const sps::RowBytes *of, int many) {
    for (int k = 0; k < many; ++k)
      if (sps::rows_overlap(x, of[k])) return true;
    return false;
  };
  if (in_any(losses, rows, 2) || in_any(losses, lists, 3) || in_any(losses, grads, 2))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: the losses overlap other arguments", what);
  if (in_any(grads[0], lists, 3) || in_any(grads[1], lists, 3))
    return set_error(SPS_ERR_INVALID_ARGUMENT,
                     "%s: a gradient overlaps the targets, the bias or the weights", what);
  if (!(temperature >= 1e-6f && temperature <= 1e6f))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: temperature must be in [1e-6, 1e6]", what);
  if (n > 0 && (!targets || !loss))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL targets or loss", what);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (n == 0 || m == 0) {  // no logits: nothing is learned
    if (n > 0) launch_zero(loss, 1, n * 4, n * 4, s);
    if (grad_queries) launch_zero(grad_queries, n, d * sg, ld_queries * sg, s);
    if (grad_items) launch_zero(grad_items, m, d * sg, ld_items * sg, s);
    return sps::launch_status(what);
  }
  const Shape h = shape_of(queries, items, grad_queries != nullptr, grad_items != nullptr);
  const Layout L = layout_of(h);
  if (!workspace) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL workspace", what);
  if (workspace_bytes < L.total)
    return set_error(SPS_ERR_WORKSPACE_TOO_SMALL, "%s: need %zu bytes, got %zu", what, L.total,
                     workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", what);
  const sps::RowBytes used{workspace, 1, (int64_t)L.total, (int64_t)L.total};
  if (in_any(used, rows, 2) || in_any(used, lists, 3) || in_any(used, grads, 2) || in_any(used, &losses, 1))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: the workspace overlaps other arguments", what);
  uint8_t *const ws = static_cast<uint8_t *>(workspace);
  const int np = planes(h);
  const bool wide = np > 1, grad = h.gq || h.gi;
  float *const scale = h.dtype != SPS_BF16 && grad ? reinterpret_cast<float *>(ws + L.scale) : nullptr;
  // operands: as they lie, or laid out with 16-byte rows; transposed for the products
  sps::LayBoth both{};
  both.scale = {row_weights, targets, n, m, scale};
  const auto lay = [&](int side, const sps_scores *x, bool pack, size_t packed, bool turn, size_t turned,
                       sps::RowMask mask) {
    GemmOperand o{static_cast<const uint8_t *>(x->data), x->n_rows, x->ld * 2, 0};
    sps::LayArgs &a = both.side[side];
    a.x = x->data;
    a.ld = x->ld;
    a.rows = x->n_rows;
    a.cols = x->n_cols;
    if (pack) {
      a.packed = reinterpret_cast<uint16_t *>(ws + packed);
      a.ld_p = packed_ld(h);
      a.plane_p = a.ld_p * a.rows;
      o = {ws + packed, a.rows, a.ld_p * 2, a.plane_p * 2};
    }
    if (turn) {
      a.turned = reinterpret_cast<uint16_t *>(ws + turned);
      a.ld_t = turned_ld(a.rows);
      a.plane_t = a.ld_t * a.cols;
    }
    a.mask = mask;
    if (wide) {
      a.row_scale = reinterpret_cast<float *>(ws + (side ? L.rows_i : L.rows_q));
      a.tops = reinterpret_cast<float *>(ws + (side ? L.tops_i : L.tops_q));
    }
    return o;
  };
  const GemmOperand oq = lay(0, queries, h.pack_q, L.packed_q, h.gi, L.turned_q,
                             {targets, row_weights, m, nullptr});
  const GemmOperand oi = lay(1, items, h.pack_i, L.packed_i, h.gq, L.turned_i, {nullptr, nullptr, 0, bias});

  if (wide) {
    const sps::MaxBoth max{{both.side[0], both.side[1]}};
    hipLaunchKernelGGL(sps::ce_max_kernel, dim3(2 * sps::kMaxBlocks),
                       dim3(64 * sps::kMaxWaves), 0, s, max);
  }
  launch_lay(h.dtype, &both, s);

  const float alpha = (float)(1.0 / (double)temperature);
  const int64_t k_logits = up(d, 8) * 2;
  for (int64_t r0 = 0; r0 < n; r0 += h.piece) {
    const int64_t rows = n - r0 < h.piece ? n - r0 : h.piece;
    sps::LogitArgs a{};
    a.g.q = {oq.base + r0 * oq.ld, rows, oq.ld, oq.plane};
    a.g.p = oi;
    a.g.k_bytes = k_logits;
    a.g.splits = 1;
    const double f = bias ? 1.0 / (double)temperature : 1.0;
    const double unit = bias ? sps::kLog2e : sps::kLog2e / (double)temperature;
    a.c = (float)unit;
    a.f = (float)f;
    a.f_low = (float)(f - (double)a.f);
    a.bias = bias;
    if (wide) {
      a.scale_q = both.side[0].row_scale + r0;
      a.scale_p = both.side[1].row_scale;
    }
    a.targets = targets + r0;
    a.code = grad ? ws + L.code : nullptr;
    a.ld = h.ld_g;
    a.stats = reinterpret_cast<float2 *>(ws + L.stats);
    a.blocks = h.blocks;
    a.z_target = reinterpret_cast<float *>(ws + L.z_target);
    // a last piece that is shorter: the same tiles, whose columns the statistics go by, but fewer
    sps::TilePlan plan = h.plan_l;
    plan.main_r = (int32_t)ceil_div(rows, plan.size());
    if (wide) launch_logits<sps::OpF32, sps::CodeF32>(plan, a, s);
    else if (h.dtype == SPS_F16) launch_logits<sps::OpF16, sps::CodeF16>(plan, a, s);
    else launch_logits<sps::OpBf16, sps::CodeBf16>(plan, a, s);

    sps::GradArgs c{};
    c.stats = a.stats;
    c.rows = rows;
    c.cols = m;
    c.blocks = (int32_t)h.blocks;
    c.block = h.block;
    c.z_target = a.z_target;
    c.unit = unit;
    c.weights = row_weights ? row_weights + r0 : nullptr;
    c.targets = a.targets;
    c.scale = scale;
    c.loss = loss + r0;
    if (!grad) {
      hipLaunchKernelGGL(sps::ce_loss_kernel, dim3((uint32_t)ceil_div(rows, 16)), dim3(256), 0, s, c);
      continue;
    }
    c.code = a.code;
    c.ld = h.ld_g;
    c.g = reinterpret_cast<uint16_t *>(ws + L.g);
    c.plane_g = h.piece * h.ld_g;
    c.factor = reinterpret_cast<float *>(ws + L.factor);
    launch_grad(h.dtype, c, s);

    sps::ProductsArgs p{};
    if (h.gq) {
      sps::ProductArgs &x = p.queries;
      x.g.q = {reinterpret_cast<const uint8_t *>(c.g), rows, h.ld_g * 2, c.plane_g * 2};
      x.g.p = {ws + L.turned_i, d, turned_ld(m) * 2, turned_ld(m) * d * 2};
      x.g.k_bytes = up(m, 64) * 2;
      x.part = reinterpret_cast<float *>(ws + L.part_q);
      x.out = static_cast<uint8_t *>(grad_queries) + r0 * ld_queries * sg;
      x.ld = ld_queries;
      x.dtype = grad_dtype;
      x.alpha = alpha;
      x.scale = scale;
      x.tops = wide ? both.side[1].tops : nullptr;
      x.mask = {c.factor, nullptr};
    }
    if (h.gi) {
      sps::ProductArgs &x = p.items;
      x.g.q = {reinterpret_cast<const uint8_t *>(c.g), m, h.ld_g * 2, c.plane_g * 2};
      x.g.k_rows = rows;
      x.g.p = {ws + L.turned_q + r0 * 2, d, turned_ld(n) * 2, turned_ld(n) * d * 2};
      x.g.k_bytes = up(rows, 8) * 2;
      float *const sum = reinterpret_cast<float *>(ws + L.sum_i);
      x.part = reinterpret_cast<float *>(ws + L.part_i);
      x.before = r0 > 0 ? sum : nullptr;
      if (r0 + rows == n) {
        x.out = grad_items;
        x.ld = ld_items;
        x.dtype = grad_dtype;
        x.alpha = alpha;
        x.scale = scale;
        x.tops = wide ? both.side[0].tops : nullptr;
        x.mask = {nullptr, bias};
      } else {  // as they are
        x.out = sum;
        x.ld = d;
        x.dtype = SPS_F32;
        x.alpha = 1.0f;
      }
    }
    launch_products(h.dtype, plan_products(h, rows), &p, s);
  }
  return sps::launch_status(what);
}

}  // extern "C"
