// sps_int8.hip -- dense rows in 8 bits: to integers and back, and the products
// of two sets of such rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sps_gemm.h"

namespace sps {

// ---------------------------------------------------------------------------
// rows to 8 bits

// 16 bytes of values on any boundary of T, one load or store: as an array of
// values (Vec) the compiler takes it in parts (500,000 x 200 bf16 97 us to 8
// bits instead of 70, 100,000 x 1024 float32 133 us back instead of 96).
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2), may_alias));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4), may_alias));
template <typename T>
using Sixteen = std::conditional_t<sizeof(T) == 4, u32x4_at4, u32x4_at2>;
template <typename T>
__device__ __forceinline__ u32x4 load16(const T *x) {
  return *reinterpret_cast<const Sixteen<T> *>(x);
}
template <typename T>
__device__ __forceinline__ void store16(T *x, u32x4 v) {
  *reinterpret_cast<Sixteen<T> *>(x) = v;
}
template <typename T>
__device__ __forceinline__ float value16(u32x4 v, int e) {
  const uint32_t w = v[e * (int)sizeof(T) / 4];
  if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w);
  else return to_f32(__builtin_bit_cast(T, (uint16_t)(w >> (16 * (e & 1)))));
}

struct QuantArgs {
  const void *x;
  int64_t ld;  // elements
  int64_t n_rows, dim;
  int8_t *q;
  int64_t ld_q;
  float *scales;
};

// The nearest integer of 127 x / amax, ties to even. y is within 3e-5 of the
// quotient; only where that leaves the side of a half open are the exact
// 254 |x| and (2 h + 1) amax compared, which float64 holds without rounding.
__device__ __forceinline__ int32_t nearest_int8(float x, float y, float amax) {
  const float k = rintf(y);
  if (__builtin_expect(fabsf(y - k) > 0.4999f, 0)) {
    const float h = floorf(fabsf(y));
    const double d = 254.0 * (double)fabsf(x) - (2.0 * (double)h + 1.0) * (double)amax;
    const int32_t m = (int32_t)h + (d > 0.0 || (d == 0.0 && ((int32_t)h & 1)));
    return x < 0.0f ? -m : m;
  }
  return (int32_t)k;
}

// L lanes a row, so that most rows fit the four vectors that a lane keeps in
// registers between the maximum and the integers and few lanes are left over;
// what does not fit is read again (from the caches). 500,000 x 333 float32 in 151
// to 173 us, 5.5 to 4.8 TB/s, bound by memory; bf16 in 132 to 158 and fp16 in 134
// to 144, 3.8 to 3.2 TB/s, by their instructions, a wave's 4 cycles each (two vectors a lane: 182, eight spill: 275; 64 lanes for
// every row, before: 230 instead of 144).
constexpr int kQuantKeep = 4;
template <typename T, int L>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
  constexpr int V = kVec<T>;
  const int lane = threadIdx.x % L;
  const int64_t r = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const bool there = r < a.n_rows;
  const T *const x = static_cast<const T *>(a.x) + (there ? r : 0) * a.ld;
  const int dim = (int)a.dim, whole = dim / V;  // whole vectors; the rest of the row is one short one
  const int tail = dim - whole * V, vecs = whole + (tail > 0);
  const auto fetch = [&](int v) {
    u32x4 t{};
    if (v < whole) t = load16(x + v * V);
    else if (v == whole) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < tail) {
          if constexpr (sizeof(T) == 4) t[e] = __builtin_bit_cast(uint32_t, x[v * V + e]);
          else t[e / 2] |= (uint32_t)x[v * V + e].u << (16 * (e & 1));
        }
    }
    return t;
  };
  u32x4 keep[kQuantKeep] = {};
  uint32_t top = 0;  // bits of magnitudes: their order, NaN above infinity
  const auto see = [&](u32x4 t) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const uint32_t b = __builtin_bit_cast(uint32_t, value16<T>(t, e)) & 0x7fffffffu;
      top = b > top ? b : top;
    }
  };
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i)
    if (L * i < vecs) keep[i] = fetch(lane + L * i);
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i)
    if (L * i < vecs) see(keep[i]);
  for (int v = lane + L * kQuantKeep; v < vecs; v += L) see(fetch(v));
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    const uint32_t b = (uint32_t)__shfl_xor((int)top, o, 64);
    top = b > top ? b : top;
  }
  if (!there) return;
  const float amax = __builtin_bit_cast(float, top);
  const bool finite = top < 0x7f800000u;
  // rows of very small values are taken 2^64 times as large: 127 / amax must not overflow
  const float up = amax < 0x1p-60f ? 0x1p64f : 1.0f;
  const float inv = finite && top ? 127.0f / (amax * up) : 0.0f;
  int8_t *const q = a.q + r * a.ld_q;
  const int room = (dim + 15) & ~15;  // up to there the row is filled with zeros
  const auto put = [&](int v, u32x4 t) {
    if (v * V >= room) return;
    uint32_t w[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      w[j] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = value16<T>(t, 4 * j + e);
        const int32_t k = inv > 0.0f ? nearest_int8(f, f * up * inv, amax) : 0;
        w[j] |= (uint32_t)(k & 255) << (8 * e);
      }
    }
    __builtin_memcpy(__builtin_assume_aligned(q + v * V, V), w, V);
  };
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i)
    if (L * i * V < room) put(lane + L * i, keep[i]);
  for (int v = lane + L * kQuantKeep; v * V < room; v += L) put(v, fetch(v));
  if (lane == 0) a.scales[r] = finite ? amax / 127.0f : __builtin_nanf("");
}

struct DequantArgs {
  const int8_t *q;
  int64_t ld_q;
  const float *scales;
  int64_t n_rows, dim;
  void *out;
  int64_t ld;  // elements
};

// L lanes a row, 16 bytes of values a lane and step, kDequantAhead steps' bytes
// loaded together. Bound by memory: 100,000 x 1024 float32 in 88 us, 5.8 TB/s,
// 500,000 x 333 in 217, 3.8 TB/s (rows off their 16-byte boundaries; with lanes
// that start on them 250), bf16 in 108, 4.6 TB/s. One step at a time: 96, 227 and
// 135 us, four: 86, 216 and 109, a lane a vector: 88, 217 and 138.
constexpr int kDequantAhead = 2;
template <typename T, int L>
__global__ __launch_bounds__(256) void dequantize_rows_kernel(DequantArgs a) {
  constexpr int V = kVec<T>;
  const int64_t r = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (r >= a.n_rows) return;
  const int dim = (int)a.dim;
  const int8_t *const q = a.q + r * a.ld_q;
  const float s = a.scales[r];
  T *const out = static_cast<T *>(a.out) + r * a.ld;
  typedef int8_t Bytes __attribute__((ext_vector_type(V)));
  const auto put = [&](int c, Bytes w) {
    T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = from_f32<T>((float)w[e] * s);
    if (c + V <= dim) {
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) v[j] = __builtin_bit_cast(uint32_t, t[j]);
        else v[j] = (uint32_t)t[2 * j].u | (uint32_t)t[2 * j + 1].u << 16;
      }
      store16(out + c, v);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e < dim) out[c + e] = t[e];
    }
  };
  for (int c = (int)(threadIdx.x % L) * V; c < dim; c += kDequantAhead * L * V) {
    Bytes w[kDequantAhead];  // the row's bytes reach to the next multiple of 16
#pragma unroll
    for (int i = 0; i < kDequantAhead; ++i)
      if (c + i * L * V < dim) w[i] = *reinterpret_cast<const Bytes *>(q + c + i * L * V);
#pragma unroll
    for (int i = 0; i < kDequantAhead; ++i)
      if (c + i * L * V < dim) put(c + i * L * V, w[i]);
  }
}

// ---------------------------------------------------------------------------
// scores

struct Int8Args {
  GemmArgs g;  // q: queries, p: items
  const float *scale_q, *scale_p;
  void *out;
  int64_t ld;  // elements
};

// The integers' sums are exact; a score is rounded as an integer above 2^24,
// by either scale and to its type. The smaller scale first: a sum times it
// overflows only where the score does.
__device__ __forceinline__ float score_of(int32_t sum, float sq, float sp) {
  const bool less = sq < sp;
  return (float)sum * (less ? sq : sp) * (less ? sp : sq);  // either scale's NaN stays
}

template <typename T, bool STREAM, int TC, int TR, int WC, int WR>
__global__ __launch_bounds__(64 * WC * WR) void int8_scores_kernel(Int8Args a) {
  using Tile = GemmTile<OpI8, TC, TR, WC, WR>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tile::kLds];
  Tile t(a.g, lds);
  const int64_t rows = a.g.q.rows, cols = a.g.p.rows;
  float sp[Tile::kFragC][4], sq[Tile::kFragR];
  const auto take = [&] {
    t.of_columns(a.scale_p, 0.0f, sp);
#pragma unroll
    for (int j = 0; j < Tile::kFragR; ++j) {
      const int64_t r = t.at.row0 + t.row_of(j);
      sq[j] = a.scale_q[r < rows ? r : rows - 1];
    }
  };
  const auto put_all = [&](auto whole) {
#pragma unroll
    for (int j = 0; j < Tile::kFragR; ++j) {
      typename QuadOf<T>::Bits w[Tile::kFragC];
#pragma unroll
      for (int i = 0; i < Tile::kFragC; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = score_of(t.acc[i][j][e], sq[j], sp[i][e]);
        w[i] = quad_of<T>(v);
      }
      t.template store<T, whole.value, STREAM>(j, w, static_cast<T *>(a.out), a.ld, rows, cols);
    }
  };
  const auto put = [&] {
    const bool whole = t.full();
    if (whole) put_all(std::true_type{});
    else put_all(std::false_type{});
    return whole;
  };
  gemm_tiles<Tile::template kStores<T>>(t, a.g, OpI8{}, blockIdx.x, [&] { t.clear(); }, take, put);
}

// Few queries (up to 16 NQ): bound by reading the items once. A wave takes 16
// items at a time straight from memory into a matrix instruction's operand,
// the queries lie in LDS in the order the instructions read them. 1 x 2M of 384
// dims: 152 us, 5.0 TB/s (the next items' loads behind the last products of
// these: 183), 2 or 8 loads ahead 150 or 158, of 768 dims 283 or 276 instead of
// 279, 1 x 500,000 of 200 dims 24 or 20 instead of 19.
constexpr int kFewAhead = 4;
template <typename T, int NQ>
__global__ __launch_bounds__(256) void int8_few_kernel(Int8Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int steps = (int)((a.g.k_bytes + 63) / 64);
  i32x4 *const qs = reinterpret_cast<i32x4 *>(few_lds);
  for (int i = threadIdx.x; i < steps * NQ * 64; i += 256) {
    const int l = i & 63, f = (i >> 6) % NQ, s = (i >> 6) / NQ;
    const int64_t r = f * 16 + (l & 15), k = (int64_t)s * 64 + (l >> 4) * 16;
    qs[i] = r < a.g.q.rows && k < a.g.k_bytes
                ? *reinterpret_cast<const i32x4 *>(a.g.q.base + r * a.g.q.ld + k)
                : i32x4{};
  }
  __syncthreads();
  const int64_t groups = (a.g.p.rows + 15) / 16, stride = (int64_t)gridDim.x * 4;
  // kFewAhead loads of items at a time, and as many of what comes next, be it the next items', on
  // their way while these are multiplied
  i32x4 p[kFewAhead] = {}, next[kFewAhead] = {};
  const auto fetch = [&](int64_t g, int s, i32x4 (&to)[kFewAhead]) {
    const int64_t item = g * 16 + (lane & 15), last = a.g.p.rows - 1;
    const uint8_t *const row = a.g.p.base + (item < last ? item : last) * a.g.p.ld;
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u) {
      const int64_t k = (int64_t)(s + u) * 64 + (lane >> 4) * 16;
      // past the row's end the queries are zeros: any finite bytes do
      if (s + u < steps) to[u] = *reinterpret_cast<const i32x4 *>(row + (k < a.g.k_bytes ? k : 0));
    }
  };
  int64_t g = (int64_t)blockIdx.x * 4 + wave;
  if (g >= groups) return;
  i32x4 acc[NQ] = {};
  int s = 0;
  fetch(g, 0, p);
  for (;;) {
    const bool ends = s + kFewAhead >= steps;
    const int64_t g_next = ends ? g + stride : g;
    const int s_next = ends ? 0 : s + kFewAhead;
    if (g_next < groups) fetch(g_next, s_next, next);
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u)
      if (s + u < steps)
#pragma unroll
        for (int f = 0; f < NQ; ++f) acc[f] = OpI8::mma(p[u], qs[((s + u) * NQ + f) * 64 + lane], acc[f]);
    if (ends) {
      const int64_t c0 = g * 16 + (lane >> 4) * 4;
      float sp[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sp[e] = c0 + e < a.g.p.rows ? a.scale_p[c0 + e] : 0.0f;
#pragma unroll
      for (int f = 0; f < NQ; ++f) {
        const int64_t r = f * 16 + (lane & 15);
        if (r < a.g.q.rows) {
          const float sq = a.scale_q[r];
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = score_of(acc[f][e], sq, sp[e]);
          put_four<T>(static_cast<T *>(a.out) + r * a.ld, c0, a.g.p.rows, v);
        }
        acc[f] = i32x4{};
      }
      if (g_next >= groups) break;
    }
    g = g_next;
    s = s_next;
    for (int u = 0; u < kFewAhead; ++u) p[u] = next[u];
  }
}

}  // namespace sps

using sps::set_error;

namespace {

constexpr int64_t kMax31 = 2147483647ll;
constexpr int64_t kInt8MaxDim = 131072;  // 127^2 dim stays below 2^31

sps_status check_rows8(const sps_int8_rows *x, const char *what) {
  if (!x) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL rows", what);
  if (x->n_rows < 0 || x->dim < 1)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: negative rows or no dims", what);
  if (x->n_rows >= kMax31) return set_error(SPS_ERR_OVERFLOW, "%s: rows must be below 2^31", what);
  if (x->dim > kInt8MaxDim)
    return set_error(SPS_ERR_UNSUPPORTED, "%s: at most %lld dims", what, (long long)kInt8MaxDim);
  if (x->ld < x->dim || x->ld % 16)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: ld %lld, a multiple of 16 from %lld on", what,
                     (long long)x->ld, (long long)x->dim);
  if (x->ld > sps::kMostBytes / 256)
    return set_error(SPS_ERR_OVERFLOW, "%s: ld must be below 2^23", what);
  if (x->n_rows > 0 && (!x->values || !x->scales))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL values or scales", what);
  if (reinterpret_cast<uintptr_t>(x->values) % 16)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: values must be 16-byte aligned", what);
  if (reinterpret_cast<uintptr_t>(x->scales) % 4)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: scales not aligned to their elements", what);
  return SPS_OK;
}

// Lanes a row: the fewest whose `each` vectors hold it.
template <typename T, template <typename, int> class Launch, class Args>
void launch_lanes(const Args &a, int each, hipStream_t s) {
  const int64_t lanes = sps::ceil_div(sps::ceil_div(a.dim, sps::kVec<T>), each);
  if (lanes <= 4) Launch<T, 4>::go(a, s);
  else if (lanes <= 8) Launch<T, 8>::go(a, s);
  else if (lanes <= 16) Launch<T, 16>::go(a, s);
  else if (lanes <= 32) Launch<T, 32>::go(a, s);
  else Launch<T, 64>::go(a, s);
}
template <typename T, int L>
struct Quantize {
  static void go(const sps::QuantArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((sps::quantize_rows_kernel<T, L>), dim3((uint32_t)sps::ceil_div(a.n_rows, 256 / L)),
                       dim3(256), 0, s, a);
  }
};
template <typename T, int L>
struct Dequantize {
  static void go(const sps::DequantArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((sps::dequantize_rows_kernel<T, L>), dim3((uint32_t)sps::ceil_div(a.n_rows, 256 / L)),
                       dim3(256), 0, s, a);
  }
};

template <typename T, int NQ>
void launch_few(const sps::Int8Args &a, hipStream_t s) {
  const size_t lds = (size_t)((a.g.k_bytes + 63) / 64) * NQ * 1024;
  int64_t blocks = sps::ceil_div(sps::ceil_div(a.g.p.rows, 16), 4);
  if (blocks > 2048) blocks = 2048;
  hipLaunchKernelGGL((sps::int8_few_kernel<T, NQ>), dim3((uint32_t)blocks), dim3(256), lds, s, a);
}

template <typename T, int TC, int TR, int WC, int WR>
void launch_tiles(const sps::TilePlan &plan, sps::Int8Args &a, hipStream_t s) {
  plan.give(&a.g);
  const dim3 grid(plan.grid()), block(64 * WC * WR);
  // rows on whole lines: so is every tile's run of them
  if (((uint64_t)(uintptr_t)a.out | (uint64_t)a.ld * sizeof(T)) % 128 == 0)
    hipLaunchKernelGGL((sps::int8_scores_kernel<T, true, TC, TR, WC, WR>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((sps::int8_scores_kernel<T, false, TC, TR, WC, WR>), grid, block, 0, s, a);
}

// Queries in LDS. Few queries read the items once, in the order they lie in; more have the tiles,
// whose rows of scores are put together before they are stored. 384 dims, few against tiles: 1 x 2M
// 152 against 240 us, 16 x 2M 196 against 241, 32 x 500,000 45 against 58, 64 x 500,000 89 against 63.
constexpr int64_t kFewLds = 64 * 1024;

template <typename T>
void launch_scores(sps::Int8Args &a, hipStream_t s) {
  const int64_t n = a.g.q.rows, steps = (a.g.k_bytes + 63) / 64;
  if (n <= 16 && steps * 1024 <= kFewLds) return launch_few<T, 1>(a, s);
  if (n <= 32 && steps * 2048 <= kFewLds) return launch_few<T, 2>(a, s);
  const sps::TilePlan plan =
      sps::plan_tiles(n, a.g.p.rows, sps::ceil_div(a.g.k_bytes, sps::kStep), 1);
  if (plan.big) launch_tiles<T, 256, 256, 2, 4>(plan, a, s);
  else launch_tiles<T, 128, 128, 2, 2>(plan, a, s);
}

}  // namespace

extern "C" {

sps_status sps_quantize_rows(const sps_scores *x, int8_t *values, int64_t ld, float *scales,
                             void *stream) {
  const char *what = "sps_quantize_rows";
  sps_status st = sps::check_scores(x, what);
  if (st != SPS_OK) return st;
  const sps_int8_rows out{values, scales, x->n_rows, x->n_cols, ld};
  st = check_rows8(&out, what);
  if (st == SPS_OK) st = sps::check_grid(sps::ceil_div(x->n_rows, 4), 256, what);
  if (st != SPS_OK) return st;
  if (x->n_rows == 0) return SPS_OK;
  const int64_t size = sps::dtype_size(x->dtype);
  const sps::RowBytes rows{x->data, x->n_rows, x->n_cols * size, x->ld * size};
  const sps::RowBytes integers{values, x->n_rows, (x->n_cols + 15) & ~15ll, ld};
  const sps::RowBytes of_scales{scales, 1, x->n_rows * 4, x->n_rows * 4};
  if (sps::rows_overlap(rows, integers) || sps::rows_overlap(rows, of_scales) ||
      sps::rows_overlap(integers, of_scales))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: rows, integers and scales overlap", what);
  sps::QuantArgs a{x->data, x->ld, x->n_rows, x->n_cols, values, ld, scales};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (x->dtype == SPS_F32) launch_lanes<float, Quantize>(a, sps::kQuantKeep, s);
  else if (x->dtype == SPS_F16) launch_lanes<sps::f16_t, Quantize>(a, sps::kQuantKeep, s);
  else launch_lanes<sps::bf16_t, Quantize>(a, sps::kQuantKeep, s);
  return sps::launch_status(what);
}

sps_status sps_dequantize_rows(const sps_int8_rows *x, void *out, int32_t dtype, int64_t ld_out,
                               void *stream) {
  const char *what = "sps_dequantize_rows";
  sps_status st = check_rows8(x, what);
  if (st != SPS_OK) return st;
  const sps_scores view{out, dtype, x->n_rows, x->dim, ld_out, 0};
  st = sps::check_scores(&view, what);
  if (st == SPS_OK) st = sps::check_grid(sps::ceil_div(x->n_rows, 4), 256, what);
  if (st != SPS_OK) return st;
  if (x->n_rows == 0) return SPS_OK;
  const int64_t size = sps::dtype_size(dtype);
  const sps::RowBytes o{out, x->n_rows, x->dim * size, ld_out * size};
  if (sps::rows_overlap(o, {x->values, x->n_rows, (x->dim + 15) & ~15ll, x->ld}) ||
      sps::rows_overlap(o, {x->scales, 1, x->n_rows * 4, x->n_rows * 4}))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: the output overlaps the 8-bit rows", what);
  sps::DequantArgs a{x->values, x->ld, x->scales, x->n_rows, x->dim, out, ld_out};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SPS_F32) launch_lanes<float, Dequantize>(a, sps::kDequantAhead, s);
  else if (dtype == SPS_F16) launch_lanes<sps::f16_t, Dequantize>(a, sps::kDequantAhead, s);
  else launch_lanes<sps::bf16_t, Dequantize>(a, sps::kDequantAhead, s);
  return sps::launch_status(what);
}

sps_status sps_int8_scores(const sps_int8_rows *queries, const sps_int8_rows *items, void *out,
                           int32_t dtype, int64_t ld_out, void *stream) {
  const char *what = "sps_int8_scores";
  sps_status st = check_rows8(queries, what);
  if (st == SPS_OK) st = check_rows8(items, what);
  if (st != SPS_OK) return st;
  if (queries->dim != items->dim)
    return set_error(SPS_ERR_DIM_MISMATCH, "%s: queries have %lld dims, items %lld", what,
                     (long long)queries->dim, (long long)items->dim);
  const sps_scores view{out, dtype, queries->n_rows, items->n_rows, ld_out, 0};
  st = sps::check_scores(&view, what);
  // a workgroup of 256 threads for 128 x 128 scores at the least
  if (st == SPS_OK)
    st = sps::check_grid(sps::ceil_div(queries->n_rows, 128) * sps::ceil_div(items->n_rows, 128),
                         512, what);
  if (st != SPS_OK) return st;
  if (queries->n_rows == 0 || items->n_rows == 0) return SPS_OK;
  const int64_t size = sps::dtype_size(dtype), k = (queries->dim + 15) & ~15ll;
  const sps::RowBytes o{out, queries->n_rows, items->n_rows * size, ld_out * size};
  if (sps::rows_overlap(o, {queries->values, queries->n_rows, k, queries->ld}) ||
      sps::rows_overlap(o, {items->values, items->n_rows, k, items->ld}) ||
      sps::rows_overlap(o, {queries->scales, 1, queries->n_rows * 4, queries->n_rows * 4}) ||
      sps::rows_overlap(o, {items->scales, 1, items->n_rows * 4, items->n_rows * 4}))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: the scores overlap the rows", what);
  sps::Int8Args a{};
  a.g.q = {reinterpret_cast<const uint8_t *>(queries->values), queries->n_rows, queries->ld, 0};
  a.g.p = {reinterpret_cast<const uint8_t *>(items->values), items->n_rows, items->ld, 0};
  a.g.k_bytes = k;
  a.scale_q = queries->scales;
  a.scale_p = items->scales;
  a.out = out;
  a.ld = ld_out;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SPS_F32) launch_scores<float>(a, s);
  else if (dtype == SPS_F16) launch_scores<sps::f16_t>(a, s);
  else launch_scores<sps::bf16_t>(a, s);
  return sps::launch_status(what);
}

}  // extern "C"
