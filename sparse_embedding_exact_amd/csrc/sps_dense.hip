// sps_dense.hip -- softmax cross entropy of dense queries over dense items, and
// its gradients, without the logits.
//
// With z = x . w / tau + b and G = weight / tau (softmax(z) - onehot(target)):
//   loss = lse(z) - z_target,  grad x = G w,  grad w = G^T x.
// Three matrix products, the least there is, for a piece of the rows at a time:
//   1. logits: a tile's z in registers; its rows' maxima and sums of
//      exponentials go to `stats`, and e^(z - max) in 16 bits to `code`;
//   2. sums: a row's log-sum-exp and loss from its blocks' statistics;
//   3. gradient of the logits: code to G in place, and G transposed;
//   4. two products with G, whose k (items, or rows) lies in one run.
// Code: a 16-bit float below the block's maximum, with 3 or 2 bits more than
// G keeps when it is rounded to enter the matrix instructions, so z is not
// computed twice. G's own column at the
// target is 1 - p from the loss, never p - 1 of a rounded p.
// fp16: G is held 2^k times as large, 2^k the power of two that takes the
// largest weight to [2^14, 2^15), so that p down to 2^-29 keeps all its bits.
// float32: operands and G stand as three bf16 planes, their values' 24 bits;
// six products of planes leave out what is below 2^-24 of a product.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sps_gemm.h"

namespace sps {

// ---------------------------------------------------------------------------
// operands

// 16-bit planes of a value: itself, or a float32 as hi + mid + low in bf16.
template <typename T>
constexpr int kPlanes = 1;
template <>
constexpr int kPlanes<float> = 3;

__device__ __forceinline__ void split(f16_t x, uint16_t o[1]) { o[0] = x.u; }
__device__ __forceinline__ void split(bf16_t x, uint16_t o[1]) { o[0] = x.u; }
// Nearest bf16 of what is left each time: the last one is exact. Infinities and
// NaN, and what rounds to infinity, stand in the leading plane.
__device__ __forceinline__ void split(float x, uint16_t o[3]) {
  const bf16_t hi = from_f32<bf16_t>(x);
  const float h = to_f32(hi);
  const bool fine = fabsf(h) < __builtin_inff();
  const float r = fine ? x - h : 0.0f;
  const bf16_t mid = from_f32<bf16_t>(r);
  o[0] = hi.u;
  o[1] = mid.u;
  o[2] = from_f32<bf16_t>(r - to_f32(mid)).u;
}

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
};

// Tiles of 64 x 64 through LDS; bound by memory. Planes in elements.
template <typename T>
__global__ __launch_bounds__(256) void lay_kernel(LayArgs a) {
  constexpr int NP = kPlanes<T>;
  __shared__ uint16_t tile[NP][64][66];
  const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T *const x = static_cast<const T *>(a.x);
  for (int i = wave; i < 64; i += 4) {
    const int64_t r = r0 + i, c = c0 + lane;
    uint16_t v[NP] = {};
    if (r < a.rows && c < a.cols) split(x[r * a.ld + c], v);
    if (a.packed && r < a.rows && c < a.ld_p)
#pragma unroll
      for (int p = 0; p < NP; ++p) a.packed[p * a.plane_p + r * a.ld_p + c] = v[p];
    if (!a.turned) continue;
    const bool out = r < a.rows && a.mask.out(r);
#pragma unroll
    for (int p = 0; p < NP; ++p) tile[p][i][lane] = out ? (uint16_t)0 : v[p];
  }
  if (!a.turned) return;
  __syncthreads();
  for (int i = wave; i < 64; i += 4) {
    const int64_t c = c0 + i, r = r0 + lane;
    if (c < a.cols && r < a.ld_t)
#pragma unroll
      for (int p = 0; p < NP; ++p) a.turned[p * a.plane_t + c * a.ld_t + r] = tile[p][lane][i];
  }
}

// ---------------------------------------------------------------------------
// 1. logits

// How e^(z - max) is kept, in units of 2^-kShift, so that small ones stay
// normal numbers.
// bf16: as fp16 (an error of 2^-12 where G is rounded by 2^-9).
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
// fp16: float32's own bits of p 2^-112 but the last 11: 4 bits of exponent, 12
// of mantissa (an error of 2^-13 where G is rounded by 2^-12), running out
// gradually below 2^-14.
struct CodeF16 {
  using Word = uint16_t;
  static constexpr int kShift = 0;
  static __device__ __forceinline__ uint32_t one(float p) {
    return (__builtin_bit_cast(uint32_t, p * 0x1p-112f) + 0x400u) >> 11;
  }
  static __device__ __forceinline__ uint32_t two(float a, float b) { return one(a) | one(b) << 16; }
  static __device__ __forceinline__ float value(uint32_t w) {
    return __builtin_bit_cast(float, w << 11) * 0x1p112f;
  }
};
struct CodeF32 {
  using Word = float;
  static constexpr int kShift = 0;
};

struct LogitArgs {
  GemmArgs g;         // q: the piece's queries, p: items
  float c;            // log2(e) / tau: everything is in powers of two
  const float *bias;  // nullable
  const int32_t *targets;
  void *code;  // nullable: uint16 (float32: float) [rows][ld]
  int64_t ld;
  float2 *stats;  // [block of columns][rows_pad]: (max, sum of 2^(z - max))
  int64_t rows_pad;
  float *z_target;
};

constexpr float kLog2e = 1.44269504088896340736f;

template <class Op, class Code, int TC, int TR, int WC, int WR>
__global__ __launch_bounds__(64 * WC * WR) void ce_logits_kernel(LogitArgs a) {
  using Tile = GemmTile<Op, TC, TR, WC, WR>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tile::kLds];
  const GemmPlace at = gemm_place<Op, TC, TR>(a.g);
  Tile t;
  t.run(a.g, at.row0, at.col0, at.begin, at.end, lds);
  constexpr float kInf = __builtin_inff();
  constexpr int FC = Tile::kFragC, FR = Tile::kFragR;
  const int64_t cols = a.g.p.rows;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t first_col = at.col0 + (wave % WC) * (TC / WC);  // of this wave
  // The logits are c times the sums, and where there is a bias or an edge, what is put in their
  // place here.
  float c = a.c;
  if (a.bias || at.col0 + TC > cols) {
#pragma unroll
    for (int i = 0; i < FC; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t col = at.col0 + t.col_of(i) + e;
        const float b = col < cols ? (a.bias ? a.bias[col] * kLog2e : 0.0f) : -kInf;
#pragma unroll
        for (int j = 0; j < FR; ++j)  // a column that is struck out has no logit, whatever its item holds
          t.acc[i][j][e] = b == -kInf ? -kInf : __builtin_fmaf(t.acc[i][j][e], c, b);
      }
    c = 1.0f;
  }
  const int64_t block = first_col / (TC / WC);
  using Word = typename Code::Word;
  uint8_t *const mine = t.wave_lds(lds);
#pragma unroll
  for (int j = 0; j < FR; ++j) {
    const int64_t r = at.row0 + t.row_of(j);
    const bool there = r < a.g.q.rows;
    float top = -kInf;
#pragma unroll
    for (int i = 0; i < FC; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, t.acc[i][j][e]);
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64)) * c;
    // the target's logit, where it is one of this wave's columns
    const int first = there ? (int)(a.targets[r] - at.col0) : -1;
    if ((uint32_t)(first - (wave % WC) * (TC / WC)) < (uint32_t)(TC / WC)) {
#pragma unroll
      for (int i = 0; i < FC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (first == t.col_of(i) + e) a.z_target[r] = t.acc[i][j][e] * c;
    }
    const float base = (float)Code::kShift - (top == -kInf ? 0.0f : top);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < FC; ++i) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(t.acc[i][j][e], c, base));
        sum += p[e];
      }
      if (a.code) {
        if constexpr (sizeof(Word) == 2)
          t.template stage<Word>(mine, i, u32x2{Code::two(p[0], p[1]), Code::two(p[2], p[3])});
        else
          t.template stage<Word>(mine, i, f32x4{p[0], p[1], p[2], p[3]});
      }
    }
    if (a.code) {  // rows of codes are padded to a multiple of 64
      const int64_t r0 = at.row0 + t.rows_at(j);
      t.template store<Word>(mine, static_cast<Word *>(a.code) + r0 * a.ld + first_col, a.ld,
                             a.g.q.rows - r0, ((cols + 63) & ~63ll) - first_col);
    }
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    if (there && lane < 16 && first_col < cols)
      a.stats[block * a.rows_pad + r] = {top, sum * (1.0f / (float)(1 << Code::kShift))};
  }
}

// ---------------------------------------------------------------------------
// 2. sums

// What the gradient of a row's logits needs: 2^(z - lse2) and the row's factor
// (0: no gradient), and 1 - p of the target.
struct RowSum {
  float lse2, factor, rest;
  int32_t target;
};

struct SumArgs {
  const float2 *stats;
  int64_t rows_pad, rows, cols;
  int32_t blocks;
  const float *z_target, *weights;  // weights nullable
  const int32_t *targets;
  const float *scale;  // nullable: 1
  float *loss;
  RowSum *out;
};

// 16 rows a workgroup, 16 threads a row; sums beyond a block in float64.
__global__ __launch_bounds__(256) void ce_sum_kernel(SumArgs a) {
  __shared__ float tops[16][17];
  __shared__ double sums[16][17];
  const int i = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t r = (int64_t)blockIdx.x * 16 + i;
  float top = -__builtin_inff();
  double sum = 0.0;
  if (r < a.rows)
    for (int32_t b = g; b < a.blocks; b += 16) {
      const float2 s = a.stats[b * a.rows_pad + r];
      const float m = fmaxf(top, s.x);
      if (m == -__builtin_inff()) sum += (double)s.y;
      else
        sum = sum * (double)__builtin_amdgcn_exp2f(top - m) +
              (double)s.y * (double)__builtin_amdgcn_exp2f(s.x - m);
      top = m;
    }
  tops[i][g] = top;
  sums[i][g] = sum;
  __syncthreads();
  if (threadIdx.x >= 16 || r >= a.rows) return;
  float m = -__builtin_inff();
  for (int k = 0; k < 16; ++k) m = fmaxf(m, tops[i][k]);
  double l = 0.0;
  for (int k = 0; k < 16; ++k)
    l += m == -__builtin_inff() ? sums[i][k]
                                : sums[i][k] * (double)__builtin_amdgcn_exp2f(tops[i][k] - m);
  const int32_t t = a.targets[r];
  const bool takes = t >= 0 && t < a.cols && !(l == 0.0);  // 0: every column is struck out
  // log2 of the sum relative to the target's term
  const double d = takes ? ((double)m - (double)a.z_target[r]) + log2(l) : 0.0;
  const double loss = takes ? d * 0.69314718055994530942 : 0.0;
  a.loss[r] = (float)loss;
  if (!a.out) return;
  RowSum o;
  o.lse2 = (float)((double)m + log2(l));
  o.factor = takes ? (a.weights ? a.weights[r] : 1.0f) * (a.scale ? *a.scale : 1.0f) : 0.0f;
  o.rest = takes ? (float)-expm1(-loss) : 0.0f;
  o.target = t;
  a.out[r] = o;
}

// The power of two that takes the largest weight to [2^14, 2^15).
__global__ __launch_bounds__(1024) void ce_scale_kernel(const float *weights, const int32_t *targets,
                                                        int64_t n, int64_t m, float *scale) {
  __shared__ float tops[16];
  float top = 0.0f;
  for (int64_t r = threadIdx.x; r < n; r += 1024) {
    const int32_t t = targets[r];
    const float w = weights ? fabsf(weights[r]) : 1.0f;
    if (t >= 0 && t < m && w < __builtin_inff()) top = fmaxf(top, w);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < 16; ++i) top = fmaxf(top, tops[i]);
  int e = 14 - (int)((__builtin_bit_cast(uint32_t, top) >> 23) - 127);
  e = top == 0.0f ? 0 : (e > 100 ? 100 : (e < -100 ? -100 : e));
  *scale = __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}

// ---------------------------------------------------------------------------
// 3. gradient of the logits

struct TurnArgs {
  const void *code;  // [rows][ld]
  int64_t ld, rows, cols, rows_pad;
  const float2 *stats;
  int32_t block;  // columns of a block of statistics
  const RowSum *sums;
  uint16_t *g;  // nullable: planes of [rows][ld]; a 16-bit code's own place
  int64_t plane_g;
  uint16_t *turned;  // nullable: planes of [cols][ld_t]
  int64_t ld_t, plane_t;
};

// Tiles of 64 x 64, 16 bytes of G a thread and step both ways; bound by memory.
template <typename T, class Code>
__global__ __launch_bounds__(256) void ce_turn_kernel(TurnArgs a) {
  constexpr int NP = kPlanes<T>;
  __shared__ __attribute__((aligned(16))) uint16_t tile[NP][64][72];
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  const int i8 = (threadIdx.x & 7) * 8;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = (threadIdx.x >> 3) + 32 * h;
    const int64_t r = r0 + i, c = c0 + i8;
    uint16_t v[NP][8] = {};
    if (r < a.rows) {
      const RowSum s = a.sums[r];
      if (s.factor != 0.0f) {
        const float f =
            __builtin_amdgcn_exp2f(a.stats[(c / a.block) * a.rows_pad + r].x - s.lse2 -
                                  (float)Code::kShift) *
            s.factor;
        float p[8];
        if constexpr (sizeof(typename Code::Word) == 2) {
          const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.code) +
                                                           r * a.ld + c);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = Code::value((u[e / 2] >> (16 * (e & 1))) & 0xffffu);
        } else {
          const f32x4 *const w =
              reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.code) + r * a.ld + c);
          const f32x4 w0 = w[0], w1 = w[1];
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = e < 4 ? w0[e & 3] : w1[e & 3];
        }
        const int64_t t = s.target - c;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = c + e < a.cols ? (t == e ? -s.rest * s.factor : p[e] * f) : 0.0f;
          uint16_t o[NP];
          if constexpr (NP == 1) o[0] = from_f32<T>(x).u;
          else split(x, o);
#pragma unroll
          for (int k = 0; k < NP; ++k) v[k][e] = o[k];
        }
      }
      if (a.g)
#pragma unroll
        for (int k = 0; k < NP; ++k)
          *reinterpret_cast<uint4 *>(a.g + k * a.plane_g + r * a.ld + c) =
              *reinterpret_cast<const uint4 *>(v[k]);
    }
#pragma unroll
    for (int k = 0; k < NP; ++k)
      *reinterpret_cast<uint4 *>(&tile[k][i][i8]) = *reinterpret_cast<const uint4 *>(v[k]);
  }
  if (!a.turned) return;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = (threadIdx.x >> 3) + 32 * h;
    const int64_t c = c0 + i, r = r0 + i8;
    if (c >= a.cols || r >= a.ld_t) continue;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      uint16_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = tile[k][i8 + e][i];
      *reinterpret_cast<uint4 *>(a.turned + k * a.plane_t + c * a.ld_t + r) =
          *reinterpret_cast<const uint4 *>(v);
    }
  }
}

// ---------------------------------------------------------------------------
// 4. products with the gradient

// Which rows of the gradient are zeros whatever the sums say.
struct OutMask {
  const RowSum *sums;  // nullable: rows without a factor
  const float *bias;   // nullable: items struck out
  __device__ __forceinline__ bool out(int64_t r) const {
    return (sums && sums[r].factor == 0.0f) || (bias && bias[r] == -__builtin_inff());
  }
};

struct ProductArgs {
  GemmArgs g;
  const float *before;  // nullable: [rows][cols] sums of earlier pieces
  float *part;          // nullable: sums as they are, split z at z * stride
  int64_t stride;
  void *out;  // where part is NULL
  int64_t ld;
  int32_t dtype;
  float alpha;
  const float *scale;  // nullable: divides alpha
  OutMask mask;
};

__device__ __forceinline__ void put_typed(void *out, int32_t dtype, int64_t at, int64_t col,
                                          int64_t cols, const float v[4]) {
  if (dtype == SPS_F32) put_four<float>(static_cast<float *>(out) + at, col, cols, v);
  else if (dtype == SPS_F16) put_four<f16_t>(static_cast<f16_t *>(out) + at, col, cols, v);
  else put_four<bf16_t>(static_cast<bf16_t *>(out) + at, col, cols, v);
}

// The tile's sums, after those of earlier pieces, times alpha, to rows of T.
template <typename T, class Tile>
__device__ __forceinline__ void product_out(const ProductArgs &a, Tile &t, const GemmPlace &at,
                                            uint8_t *mine, T *out, int64_t ld, float alpha,
                                            const OutMask &mask) {
  const int64_t rows = a.g.q.rows, cols = a.g.p.rows;
#pragma unroll
  for (int j = 0; j < Tile::kFragR; ++j) {
    const int64_t r = at.row0 + t.row_of(j);
    const bool zero = r < rows && mask.out(r);
#pragma unroll
    for (int i = 0; i < Tile::kFragC; ++i) {
      const int64_t c = at.col0 + t.col_of(i);
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = t.acc[i][j][e];
        if (a.before && r < rows && c + e < cols) v[e] += a.before[r * cols + c + e];
        v[e] = zero ? 0.0f : v[e] * alpha;
      }
      t.template stage<T>(mine, i, quad_of<T>(v));
    }
    const int64_t r0 = at.row0 + t.rows_at(j), c0 = at.col0 + t.cols_at();
    t.template store<T>(mine, out + r0 * ld + c0, ld, rows - r0, cols - c0);
  }
}

template <class Op, int TC, int TR, int WC, int WR>
__global__ __launch_bounds__(64 * WC * WR) void ce_product_kernel(ProductArgs a) {
  using Tile = GemmTile<Op, TC, TR, WC, WR>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tile::kLds];
  const GemmPlace at = gemm_place<Op, TC, TR>(a.g);
  Tile t;
  t.run(a.g, at.row0, at.col0, at.begin, at.end, lds);
  const float alpha = a.scale ? a.alpha / *a.scale : a.alpha;
  uint8_t *const mine = t.wave_lds(lds);
  if (a.part) product_out<float>(a, t, at, mine, a.part + at.z * a.stride, a.g.p.rows, 1.0f, {});
  else if (a.dtype == SPS_F32)
    product_out<float>(a, t, at, mine, static_cast<float *>(a.out), a.ld, alpha, a.mask);
  else  // the rows' own type: that of the products
    product_out<typename Op::Type>(a, t, at, mine, static_cast<typename Op::Type *>(a.out), a.ld, alpha,
                                   a.mask);
}

struct JoinArgs {
  const float *part;
  int64_t stride, rows, cols;
  int32_t splits;
  void *out;
  int64_t ld;
  int32_t dtype;
  float alpha;
  const float *scale;
  OutMask mask;
};

// The splits' sums in their order, four values a thread.
__global__ __launch_bounds__(256) void ce_join_kernel(JoinArgs a) {
  const int64_t per = (a.cols + 3) / 4, all = a.rows * per;
  const float alpha = a.scale ? a.alpha / *a.scale : a.alpha;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per, c = (i - r * per) * 4;
    float v[4] = {};
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
    const bool zero = a.mask.out(r);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = zero ? 0.0f : v[e] * alpha;
    put_typed(a.out, a.dtype, r * a.ld, c, a.cols, v);
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

constexpr int64_t kMaxItems = 1ll << 22;  // a tile's rows of G stay below 2^31 bytes
constexpr int64_t kMaxDim = 1ll << 16;
// Bytes of a piece's codes and gradients (both layouts), and of statistics
// where there are no codes.
constexpr int64_t kPieceBytes = 1ll << 30;
constexpr int64_t kStatBytes = 1ll << 28;
constexpr int64_t kMaxPiece = 1ll << 20;

int64_t up(int64_t x, int64_t to) { return ceil_div(x, to) * to; }

struct Shape {
  int64_t n, m, d;
  int32_t dtype;
  bool gq, gi;  // which gradients
  bool pack_q, pack_i;
  bool big;          // tiles of 256 x 256 for the logits
  int64_t piece;     // rows of a piece, a multiple of 64
  int64_t ld_g;      // items, padded
  int32_t block;     // columns of a block of statistics
  int64_t blocks;
  sps::TilePlan plan_q, plan_i;  // of the products for the queries and the items
};

struct Layout {
  size_t scale, sums, z_target, stats, packed_q, packed_i, turned_q, turned_i, code, g, gt, part,
      sum_i, total;
};

int planes(const Shape &s) { return s.dtype == SPS_F32 ? 3 : 1; }

// Rows of 16-bit values that hold `k`, an odd number of 128 bytes: equal places
// of neighbouring rows fall into different channels of L2.
int64_t odd_ld(int64_t k) { return (ceil_div(k, 64) | 1) * 64; }
int64_t turned_ld(int64_t rows) { return odd_ld(rows); }
int64_t packed_ld(const Shape &s) {
  const int64_t ld = up(s.d, 8);
  return ld % 256 ? ld : ld + 64;
}

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
  s.ld_g = odd_ld(s.m);
  const bool grad = gq || gi;
  const int64_t each = s.dtype == SPS_F32 ? 4 + 6 * gq + 6 * gi : 2 + 2 * gi;
  s.block = 64;
  int64_t rows = grad ? kPieceBytes / (s.ld_g * each) : kStatBytes / (8 * ceil_div(s.m, 64));
  rows = rows / 256 * 256;
  if (rows < 256) rows = 256;
  if (rows > kMaxPiece) rows = kMaxPiece;
  s.piece = rows < s.n ? rows : up(s.n, 64);
  const int seg = s.dtype == SPS_F32 ? sps::kSegments : 1;
  const int64_t at_once = s.piece < s.n ? s.piece : s.n;
  const auto steps = [&](int64_t k) { return ceil_div(k * 2, sps::kStep) * seg; };
  s.big = sps::plan_tiles(at_once, s.m, steps(s.d), 1).big;
  s.block = s.big ? 128 : 64;
  s.blocks = ceil_div(s.m, s.block);
  // the queries' product: few tiles and a long k, split to fill the card
  s.plan_q = sps::plan_tiles(at_once, s.d, steps(s.m), 64);
  s.plan_i = sps::plan_tiles(s.m, s.d, steps(at_once), 1);
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
  L.z_target = take(s.piece * 4);
  L.stats = take(s.blocks * s.piece * 8);
  if (s.pack_q) L.packed_q = take(s.n * packed_ld(s) * 2 * p);
  if (s.pack_i) L.packed_i = take(s.m * packed_ld(s) * 2 * p);
  if (s.gq || s.gi) {
    L.sums = take(s.piece * (int64_t)sizeof(sps::RowSum));
    L.code = take(s.piece * s.ld_g * (p == 3 ? 4 : 2));
    if (s.gq) {
      L.turned_i = take(s.d * turned_ld(s.m) * 2 * p);
      L.g = p == 3 ? take(s.piece * s.ld_g * 6) : L.code;
      if (s.plan_q.splits > 1) L.part = take((int64_t)s.plan_q.splits * s.piece * s.d * 4);
    }
    if (s.gi) {
      L.turned_q = take(s.d * turned_ld(s.n) * 2 * p);
      L.gt = take(s.m * odd_ld(s.piece) * 2 * p);
      if (s.piece < s.n) L.sum_i = take(s.m * s.d * 4);
    }
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
  if (i->n_rows > kMaxItems)
    return set_error(SPS_ERR_UNSUPPORTED, "%s: at most %lld items", what, (long long)kMaxItems);
  const int64_t most = sps::kMostBytes / 256 / 4;  // a tile's rows in 31 bits of bytes
  if (q->ld > most || i->ld > most)
    return set_error(SPS_ERR_OVERFLOW, "%s: ld must be at most %lld", what, (long long)most);
  return sps::check_grid(ceil_div(q->n_rows, 64) * ceil_div(q->n_cols, 64), 256, what);
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

template <typename T>
void launch_lay_t(const sps::LayArgs &a, hipStream_t s) {
  const dim3 grid((uint32_t)ceil_div(a.rows, 64), (uint32_t)ceil_div(a.cols, 64));
  hipLaunchKernelGGL((sps::lay_kernel<T>), grid, dim3(256), 0, s, a);
}
void launch_lay(int32_t dtype, const sps::LayArgs &a, hipStream_t s) {
  if (dtype == SPS_F32) launch_lay_t<float>(a, s);
  else if (dtype == SPS_F16) launch_lay_t<sps::f16_t>(a, s);
  else launch_lay_t<sps::bf16_t>(a, s);
}

template <class Op, class Code>
void launch_logits(bool big, sps::LogitArgs a, hipStream_t s) {
  const int64_t t = big ? 256 : 128;
  a.g.tiles_c = (int32_t)ceil_div(a.g.p.rows, t);
  a.g.tiles_r = (int32_t)ceil_div(a.g.q.rows, t);
  const dim3 grid((uint32_t)a.g.tiles_c * (uint32_t)a.g.tiles_r);
  if (big) hipLaunchKernelGGL((sps::ce_logits_kernel<Op, Code, 256, 256, 2, 4>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((sps::ce_logits_kernel<Op, Code, 128, 128, 2, 2>), grid, dim3(256), 0, s, a);
}

template <class Op>
void launch_product(sps::TilePlan plan, sps::ProductArgs a, hipStream_t s) {
  const int64_t t = plan.big ? 256 : 128;
  a.g.splits = plan.splits;
  a.g.tiles_c = (int32_t)ceil_div(a.g.p.rows, t);
  a.g.tiles_r = (int32_t)ceil_div(a.g.q.rows, t);
  const dim3 grid((uint32_t)a.g.tiles_c * (uint32_t)a.g.tiles_r * (uint32_t)a.g.splits);
  if (plan.big) hipLaunchKernelGGL((sps::ce_product_kernel<Op, 256, 256, 2, 4>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((sps::ce_product_kernel<Op, 128, 128, 2, 2>), grid, dim3(256), 0, s, a);
}

void launch_turn(int32_t dtype, const sps::TurnArgs &a, hipStream_t s) {
  const dim3 grid((uint32_t)ceil_div(a.cols, 64), (uint32_t)ceil_div(a.rows, 64));
  if (dtype == SPS_F32)
    hipLaunchKernelGGL((sps::ce_turn_kernel<float, sps::CodeF32>), grid, dim3(256), 0, s, a);
  else if (dtype == SPS_F16)
    hipLaunchKernelGGL((sps::ce_turn_kernel<sps::f16_t, sps::CodeF16>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((sps::ce_turn_kernel<sps::bf16_t, sps::CodeBf16>), grid, dim3(256), 0, s, a);
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
  uint8_t *const ws = static_cast<uint8_t *>(workspace);
  const int np = planes(h);
  const bool wide = np == 3, grad = h.gq || h.gi;
  float *const scale = h.dtype == SPS_F16 && grad ? reinterpret_cast<float *>(ws + L.scale) : nullptr;
  if (scale)
    hipLaunchKernelGGL(sps::ce_scale_kernel, dim3(1), dim3(1024), 0, s, row_weights, targets, n, m,
                       scale);

  // operands: as they lie, or laid out with 16-byte rows; transposed for the products
  const auto lay = [&](const sps_scores *x, bool pack, size_t packed, bool turn, size_t turned,
                       sps::RowMask mask) {
    GemmOperand o{static_cast<const uint8_t *>(x->data), x->n_rows, x->ld * 2, 0};
    sps::LayArgs a{};
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
      a.mask = mask;
    }
    if (pack || turn) launch_lay(h.dtype, a, s);
    return o;
  };
  const GemmOperand oq = lay(queries, h.pack_q, L.packed_q, h.gi, L.turned_q,
                             {targets, row_weights, m, nullptr});
  const GemmOperand oi = lay(items, h.pack_i, L.packed_i, h.gq, L.turned_i, {nullptr, nullptr, 0, bias});

  const int64_t k_logits = up(d, 8) * 2;
  for (int64_t r0 = 0; r0 < n; r0 += h.piece) {
    const int64_t rows = n - r0 < h.piece ? n - r0 : h.piece;
    sps::LogitArgs a{};
    a.g.q = {oq.base + r0 * oq.ld, rows, oq.ld, oq.plane};
    a.g.p = oi;
    a.g.k_bytes = k_logits;
    a.g.splits = 1;
    a.c = (float)(1.44269504088896340736 / (double)temperature);
    a.bias = bias;
    a.targets = targets + r0;
    a.code = grad ? ws + L.code : nullptr;
    a.ld = h.ld_g;
    a.stats = reinterpret_cast<float2 *>(ws + L.stats);
    a.rows_pad = h.piece;
    a.z_target = reinterpret_cast<float *>(ws + L.z_target);
    if (wide) launch_logits<sps::OpF32, sps::CodeF32>(h.big, a, s);
    else if (h.dtype == SPS_F16) launch_logits<sps::OpF16, sps::CodeF16>(h.big, a, s);
    else launch_logits<sps::OpBf16, sps::CodeBf16>(h.big, a, s);

    sps::RowSum *const sums = grad ? reinterpret_cast<sps::RowSum *>(ws + L.sums) : nullptr;
    const sps::SumArgs b{a.stats, h.piece, rows, m, (int32_t)h.blocks, a.z_target,
                         row_weights ? row_weights + r0 : nullptr, a.targets, scale, loss + r0, sums};
    hipLaunchKernelGGL(sps::ce_sum_kernel, dim3((uint32_t)ceil_div(rows, 16)), dim3(256), 0, s, b);
    if (!grad) continue;

    sps::TurnArgs c{};
    c.code = a.code;
    c.ld = h.ld_g;
    c.rows = rows;
    c.cols = m;
    c.rows_pad = h.piece;
    c.stats = a.stats;
    c.block = h.block;
    c.sums = sums;
    if (h.gq) {
      c.g = reinterpret_cast<uint16_t *>(ws + L.g);
      c.plane_g = h.piece * h.ld_g;
    }
    if (h.gi) {
      c.turned = reinterpret_cast<uint16_t *>(ws + L.gt);
      c.ld_t = odd_ld(h.piece);
      c.plane_t = c.ld_t * m;
    }
    launch_turn(h.dtype, c, s);

    sps::ProductArgs p{};
    p.dtype = grad_dtype;
    p.alpha = (float)(1.0 / (double)temperature);
    p.scale = scale;
    if (h.gq) {
      p.g.q = {reinterpret_cast<const uint8_t *>(c.g), rows, h.ld_g * 2, c.plane_g * 2};
      p.g.p = {ws + L.turned_i, d, turned_ld(m) * 2, turned_ld(m) * d * 2};
      p.g.k_bytes = up(m, 64) * 2;
      p.out = static_cast<uint8_t *>(grad_queries) + r0 * ld_queries * sg;
      p.ld = ld_queries;
      p.mask = {sums, nullptr};
      if (h.plan_q.splits > 1) {
        p.part = reinterpret_cast<float *>(ws + L.part);
        p.stride = rows * d;
      }
      if (wide) launch_product<sps::OpF32>(h.plan_q, p, s);
      else if (h.dtype == SPS_F16) launch_product<sps::OpF16>(h.plan_q, p, s);
      else launch_product<sps::OpBf16>(h.plan_q, p, s);
      if (h.plan_q.splits > 1) {
        const sps::JoinArgs j{p.part, p.stride, rows, d, h.plan_q.splits, p.out, p.ld, grad_dtype, p.alpha,
                              scale, p.mask};
        int64_t blocks = ceil_div(rows * ceil_div(d, 4), 256);
        if (blocks > 4096) blocks = 4096;
        hipLaunchKernelGGL(sps::ce_join_kernel, dim3((uint32_t)blocks), dim3(256), 0, s, j);
      }
    }
    if (h.gi) {
      const bool last = r0 + rows == n;
      p.g.q = {ws + L.gt, m, c.ld_t * 2, c.plane_t * 2};
      p.g.p = {ws + L.turned_q + r0 * 2, d, turned_ld(n) * 2, turned_ld(n) * d * 2};
      p.g.k_bytes = up(rows, 8) * 2;
      float *const sum = reinterpret_cast<float *>(ws + L.sum_i);
      p.before = r0 > 0 ? sum : nullptr;
      p.part = last ? nullptr : sum;
      p.stride = 0;
      p.out = grad_items;
      p.ld = ld_items;
      p.mask = {nullptr, bias};
      if (wide) launch_product<sps::OpF32>(h.plan_i, p, s);
      else if (h.dtype == SPS_F16) launch_product<sps::OpF16>(h.plan_i, p, s);
      else launch_product<sps::OpBf16>(h.plan_i, p, s);
    }
  }
  return sps::launch_status(what);
}

}  // extern "C"
