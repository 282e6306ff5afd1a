// sps_distill.hip -- distillation of rows of scores from a teacher's top list
// on gfx950: the loss of every row and its gradient, over whole rows or over
// chunks of columns as they stream by.
//
// Mathematics. With c = log2(e) / temperature every exponential is 2^((x - M)
// c) for a running maximum M: the difference is taken first, so that rows of
// the type's lowest value keep a finite softmax. The columns of the teacher's
// list stay out of the running sum (a bit per column, set in LDS) and are
// added at the end from their own scores: the mass outside the list, which
// the loss with a remaining class divides by, is then a sum of its own terms
// and not a difference. From M, that sum and the listed scores a row's loss
// follows, and two factors a and b with which the gradient is b e (columns
// outside the list) and a e - p (listed), e = 2^((x - M) c).
//
// What bounds it: reading the scores for the sums, reading them again and
// writing the gradient; a score costs about ten operations.
#include <cmath>
#include <new>

#include "sps_rows.h"

namespace sps {

constexpr int kDistMaxK = 1024;   // listed entries of a row: the public limit
constexpr int kDistThreads = 256;
constexpr int kDistVpt = 32;      // scores a thread holds: one bit each of a word
constexpr int kDistTile = kDistThreads * kDistVpt;
constexpr int kSuperTiles = 8;    // tiles whose bits LDS holds at a time
constexpr int kDistFill = 1024;   // workgroups that fill the card
constexpr int kMaxSlots = 256;

struct Stat {  // sum of 2^((x - m) c) over a part of a row's unlisted columns
  double s;
  float m;
  float pad;
};

struct RowTeach {  // of a row's list
  double entropy;  // sum p log p, the remaining class's term included
  double mass;     // sum p + p_rest
  double rest;     // p_rest
  int32_t has;     // an entry takes part
  int32_t pad;
};

struct RowCoef {  // for the gradient
  double a;      // of a listed score's 2^((x - m_all) c)
  double b;      // of another score's 2^((x - m) c)
  float m_all, m;
  int32_t live;  // 0: loss and gradient are 0
  int32_t pad;
};

struct DistillDev {
  int64_t n_rows, n_cols;
  int32_t k, slots;
  float c;        // log2(e) / temperature
  double inv_tau;
  int32_t *sid;   // [rows][k]: column, -1 where the entry takes no part
  float *p;       // [rows][k]
  float *x;       // [rows][k]: the student's score of the entry
  RowTeach *teach;
  RowCoef *coef;
  Stat *stat;     // [rows][slots]
};

__device__ __forceinline__ float exp2_from(float x, float m, float c) {
  return __builtin_amdgcn_exp2f((x - m) * c);
}
// x, or -inf where bit e of `listed` is set (two operations, no branch)
__device__ __forceinline__ float strike_if(float x, uint32_t listed, int e) {
  const uint32_t mask = (uint32_t)((int32_t)(listed << (31 - e)) >> 31);
  return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & ~mask) | (0xFF800000u & mask));
}
// what a maximum of -inf (nothing but -inf yet) is subtracted as
__device__ __forceinline__ float finite_max(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// ---- reductions over a workgroup ----
// Sum of ws[0, n), n <= 16, in every lane (at = lane % 16), in a fixed order.
__device__ __forceinline__ double row16_sum(int at, int n, const double *ws) {
  double s = at < n ? ws[at] : 0.0;
  s += dpp_f64<0x111, 0xf, true>(s);  // row_shr:1
  s += dpp_f64<0x112, 0xf, true>(s);  // row_shr:2
  s += dpp_f64<0x114, 0xf, true>(s);  // row_shr:4
  s += dpp_f64<0x118, 0xf, true>(s);  // row_shr:8
  return __shfl(s, 15, 64);
}
// Sums of N doubles over NT threads, in every thread; `ws` is N x 16 doubles.
template <int NT, int N>
__device__ __forceinline__ void block_sums(double (&v)[N], double (*ws)[16]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double s = wave_total_f64(v[i]);
    if (lane == 63) ws[i][threadIdx.x >> 6] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = row16_sum(lane & 15, NT / 64, ws[i]);
  __syncthreads();
}
template <int NT>
__device__ __forceinline__ float block_max(float v, float *ws) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  const int lane = threadIdx.x & 63;
  if (lane == 0) ws[threadIdx.x >> 6] = v;
  __syncthreads();
  v = ws[lane & (NT / 64 - 1)];
#pragma unroll
  for (int o = NT / 128; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  __syncthreads();
  return v;
}

// ---- the teacher's lists ----
template <int KMAX>
struct TeachShared {
  int32_t id[KMAX];   // as given, -1 where unusable
  int32_t sid[KMAX];  // -1 where the entry takes no part
  float p[KMAX];
  double wd[3][16];
  float wf[16];
};

// By one workgroup: which entries of a row take part (an id's first
// occurrence, inside the columns, with a logit), and their masses.
template <int NT, int KMAX>
__device__ __forceinline__ RowTeach teach_row(const int32_t *__restrict__ ids,
                                              const float *__restrict__ logits, const float *lse,
                                              int k, int64_t n_cols, double inv_tau,
                                              TeachShared<KMAX> &sh) {
  const int t = threadIdx.x;
  const double given = lse ? (double)*lse : 0.0;
  for (int i = t; i < k; i += NT) {
    const int32_t v = ids[i];
    const float l = logits[i];
    sh.id[i] = v >= 0 && v < n_cols && l != -__builtin_inff() ? v : -1;
    sh.p[i] = l;
  }
  __syncthreads();
  float mx = -__builtin_inff();
  int has = 0;
  for (int i = t; i < k; i += NT) {
    const int32_t v = sh.id[i];
    int dup = v < 0;
#pragma unroll 8
    for (int j = 0; j < i; ++j) dup |= sh.id[j] == v;
    sh.sid[i] = dup ? -1 : v;
    if (!dup) {
      has = 1;
      mx = fmaxf(mx, sh.p[i]);
    }
  }
  if (!lse) mx = block_max<NT>(mx, sh.wf);
  const double shift = lse ? given : (double)finite_max(mx) * inv_tau;
  double v[3] = {0, 0, (double)has};  // sum e, sum e log e, entries
  double mine = 0;                    // of this thread's first entry
  for (int i = t; i < k; i += NT)
    if (sh.sid[i] >= 0) {
      const double x = (double)sh.p[i] * inv_tau - shift, e = exp(x);
      v[0] += e;
      v[1] += e == 0 ? 0.0 : e * x;
      if (i == t) mine = e;
    }
  block_sums<NT>(v, sh.wd);
  const double sum = v[0], scale = lse ? 1.0 : 1.0 / sum;
  // a mass below float32's range stays above 0: a listed column whose score is -inf makes the
  // loss +inf whatever its mass
  constexpr double kLeast = 1.401298464324817e-45;
  for (int i = t; i < k; i += NT) {
    if (i > t) mine = exp((double)sh.p[i] * inv_tau - shift);
    const double p = mine * scale;
    sh.p[i] = sh.sid[i] >= 0 ? (float)(p > 0 && p < kLeast ? kLeast : p) : 0.0f;
  }
  RowTeach r;
  r.has = v[2] != 0;
  r.rest = 0;
  if (lse) r.rest = sum < 1 ? 1 - sum : sum >= 1 ? 0.0 : sum;  // NaN stays
  // sum p log p: p = e scale, log p = x + log scale
  r.entropy = v[1] * scale + (lse || !r.has ? 0.0 : log(scale)) +
              (r.rest == 0 ? 0.0 : r.rest * log(r.rest));
  r.mass = lse ? sum + r.rest : 1.0 + (sum - sum);  // 1, or NaN where the logits are
  r.pad = 0;
  return r;
}

template <int NT, int KMAX>
__global__ __launch_bounds__(NT) void distill_prepare_kernel(DistillDev d,
                                                             const int32_t *__restrict__ ids,
                                                             const float *__restrict__ logits,
                                                             const float *__restrict__ lse) {
  __shared__ TeachShared<KMAX> sh;
  const int64_t row = blockIdx.x, at = row * d.k;
  const RowTeach r = teach_row<NT, KMAX>(ids + at, logits + at, lse ? lse + row : nullptr, d.k, d.n_cols,
                                   d.inv_tau, sh);
  for (int i = threadIdx.x; i < d.k; i += NT) {
    d.sid[at + i] = sh.sid[i];
    d.p[at + i] = sh.p[i];
  }
  if (threadIdx.x == 0) d.teach[row] = r;
}

// ---- the sums ----
struct ChunkArgs {
  DistillDev d;
  const void *x;
  int64_t ld, n_cols, col_begin, seg;
  int32_t splits, first;
};

// the word and bit of a column `o` columns into its tile of scores of type T
template <typename T, int NT>
__device__ __forceinline__ void bit_of(int o, int &word, int &bit) {
  constexpr int V = kVec<T>;
  const int v = o / V;
  word = v % NT;
  bit = v / NT * V + o % V;
}

// a tile's scores of this thread; columns past the end are -inf
template <typename T, int NT, int VPT>
__device__ __forceinline__ void load_tile(const T *x, int64_t base, int64_t end, float (&f)[VPT]) {
  constexpr int V = kVec<T>;
  if (base + NT * VPT <= end) {  // a whole tile: all loads in flight
    Vec<T> w[VPT / V];
#pragma unroll
    for (int v = 0; v < VPT / V; ++v)
      w[v] = *reinterpret_cast<const Vec<T> *>(x + base + ((int64_t)v * NT + threadIdx.x) * V);
#pragma unroll
    for (int i = 0; i < VPT; ++i) f[i] = to_f32(w[i / V].e[i % V]);
    return;
  }
#pragma unroll
  for (int v = 0; v < VPT / V; ++v) {
    const int64_t c = base + ((int64_t)v * NT + threadIdx.x) * V;
    if (c + V <= end) {
      const Vec<T> w = *reinterpret_cast<const Vec<T> *>(x + c);
#pragma unroll
      for (int e = 0; e < V; ++e) f[v * V + e] = to_f32(w.e[e]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        f[v * V + e] = c + e < end ? to_f32(x[c + e]) : -__builtin_inff();
    }
  }
}

// A thread's scores of a tile as they were loaded, four bytes a register: for
// 16-bit scores half the registers of their float32 values. Past the end of
// the row stands -inf.
template <typename T, int NT, int VPT>
struct RawTile {
  static constexpr int V = kVec<T>, E = 4 / (int)sizeof(T);
  uint32_t r[VPT / E];

  struct __attribute__((packed, aligned(sizeof(T)))) Quad {
    uint32_t w[4];
  };
  static __device__ __forceinline__ uint32_t bits(T v) {
    if constexpr (E == 1) return __builtin_bit_cast(uint32_t, v);
    else return v.u;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (E == 1) {
      return __builtin_bit_cast(float, r[i]);
    } else {
      T v;
      v.u = (uint16_t)(r[i / 2] >> (i % 2 * 16));
      return to_f32(v);
    }
  }
  __device__ __forceinline__ void strike(int i) {
    const uint32_t inf = bits(from_f32<T>(-__builtin_inff()));
    if constexpr (E == 1) r[i] = inf;
    else r[i / 2] = i % 2 ? (r[i / 2] & 0xFFFFu) | inf << 16 : (r[i / 2] & 0xFFFF0000u) | inf;
  }
  // columns [base, base + NT * VPT) of a row that ends at `end`
  __device__ __forceinline__ void load(const T *x, int64_t base, int64_t end) {
    if (base + NT * VPT <= end) {  // a whole tile: all loads in flight
#pragma unroll
      for (int v = 0; v < VPT / V; ++v) {
        const Quad q = *reinterpret_cast<const Quad *>(x + base + ((int64_t)v * NT + threadIdx.x) * V);
#pragma unroll
        for (int e = 0; e < 4; ++e) r[v * 4 + e] = q.w[e];
      }
      return;
    }
    const uint32_t inf = bits(from_f32<T>(-__builtin_inff()));
#pragma unroll
    for (int v = 0; v < VPT / V; ++v) {
      const int64_t c = base + ((int64_t)v * NT + threadIdx.x) * V;
      if (c + V <= end) {
        const Quad q = *reinterpret_cast<const Quad *>(x + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) r[v * 4 + e] = q.w[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t word = 0;
#pragma unroll
          for (int h = 0; h < E; ++h)
            word |= (c + e * E + h < end ? bits(x[c + e * E + h]) : inf) << (16 * h);
          r[v * 4 + e] = word;
        }
      }
    }
  }
  // Nothing derived from the scores so far is kept: a second use converts them
  // again, where the compiler would hold VPT values more across the barriers.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < VPT / E; ++i) asm volatile("" : "+v"(r[i]));
  }
  // g[...] = 2^((x - m) c) b of the tile's columns, or 0
  template <typename G>
  __device__ __forceinline__ void store(G *g, int64_t base, int64_t end, bool live, float m, float c,
                                        float b) const {
    constexpr int W = kVec<G>;
#pragma unroll
    for (int v = 0; v < VPT / V; ++v) {
      const int64_t o = base + ((int64_t)v * NT + threadIdx.x) * V;
      if (o + V <= end) {
#pragma unroll
        for (int w = 0; w < V; w += W) {
          Vec<G> q;
#pragma unroll
          for (int e = 0; e < W; ++e)
            q.e[e] = from_f32<G>(live ? exp2_from(get(v * V + w + e), m, c) * b : 0.0f);
          *reinterpret_cast<Vec<G> *>(g + o + w) = q;
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (o + e < end)
            g[o + e] = from_f32<G>(live ? exp2_from(get(v * V + e), m, c) * b : 0.0f);
      }
    }
  }
};

// A part of a row a workgroup. 10,000 x 8192 fp16: 47 us, 3.5 TB/s; bound by
// the chain of a workgroup's life (list, bits, tile, reduction), of which seven
// run on a CU, and by 13 operations a score of vector issue. One workgroup for
// many rows with the next tile loaded ahead was no faster (52 us: the list's
// loads wait for those of the tile before them).
template <typename T>
__global__ __launch_bounds__(kDistThreads) void distill_chunk_kernel(ChunkArgs a) {
  __shared__ uint32_t bits[kSuperTiles][kDistThreads];
  __shared__ double ws[kDistThreads / 64];
  __shared__ float wm[kDistThreads / 64];
  const DistillDev &d = a.d;
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x / (uint32_t)a.splits;
  const int32_t split = (int32_t)(blockIdx.x % (uint32_t)a.splits);
  const int64_t c0 = split * a.seg, c1 = c0 + a.seg < a.n_cols ? c0 + a.seg : a.n_cols;
  const T *x = static_cast<const T *>(a.x) + row * a.ld;
  const int32_t *sid = d.sid + row * d.k;
  Stat *st = d.stat + row * d.slots;
  // the first tile, the list and what came before are on their way together
  float f[kDistVpt];
  load_tile<T, kDistThreads>(x, c0, c1, f);
  Stat old{0, -__builtin_inff(), 0};
  if (!a.first) old = st[split];
  float m = -__builtin_inff();
  double s = 0;
  for (int64_t s0 = c0; s0 < c1; s0 += (int64_t)kSuperTiles * kDistTile) {
    const int64_t s1 =
        s0 + (int64_t)kSuperTiles * kDistTile < c1 ? s0 + (int64_t)kSuperTiles * kDistTile : c1;
    const int tiles = (int)((s1 - s0 + kDistTile - 1) / kDistTile);
    if (s0 > c0) __syncthreads();
    for (int i = 0; i < tiles; ++i) bits[i][t] = 0;
    __syncthreads();
    for (int i = t; i < d.k; i += kDistThreads) {
      const int32_t id = sid[i];
      const int64_t o = (int64_t)id - a.col_begin;
      if (id >= 0 && o >= s0 && o < s1) {
        int word, bit;
        bit_of<T, kDistThreads>((int)((o - s0) % kDistTile), word, bit);
        atomicOr(&bits[(o - s0) / kDistTile][word], 1u << bit);
        d.x[row * d.k + i] = to_f32(x[o]);
      }
    }
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
      if (i > 0 || s0 > c0) load_tile<T, kDistThreads>(x, s0 + (int64_t)i * kDistTile, s1, f);
      const uint32_t listed = bits[i][t];
      if (__ballot(listed != 0)) {
#pragma unroll
        for (int e = 0; e < kDistVpt; ++e) f[e] = strike_if(f[e], listed, e);
      }
      float mt = m;
#pragma unroll
      for (int e = 0; e < kDistVpt; ++e) mt = fmaxf(mt, f[e]);
      const float mf = finite_max(mt);
      float part = 0;
#pragma unroll
      for (int e = 0; e < kDistVpt; ++e) part += exp2_from(f[e], mf, d.c);
      s = s * (double)exp2_from(m, mf, d.c) + (double)part;
      m = mt;
    }
  }
  // on the first chunk, the first part clears the scores of entries that lie elsewhere
  if (a.first && split == 0)
    for (int i = t; i < d.k; i += kDistThreads) {
      const int64_t o = (int64_t)sid[i] - a.col_begin;
      if (sid[i] < 0 || o < 0 || o >= a.n_cols) d.x[row * d.k + i] = -__builtin_inff();
    }
  // a maximum and a sum of each wave, joined by one thread
  float mw = m;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mw = fmaxf(mw, __shfl_xor(mw, o, 64));
  s = wave_total_f64(s * (double)exp2_from(m, finite_max(mw), d.c));
  if ((t & 63) == 63) {
    ws[t >> 6] = s;
    wm[t >> 6] = mw;
  }
  __syncthreads();
  if (t == 0) {
    float mb = old.m;
#pragma unroll
    for (int i = 0; i < kDistThreads / 64; ++i) mb = fmaxf(mb, wm[i]);
    const float mf = finite_max(mb);
    double sb = old.s * (double)exp2_from(old.m, mf, d.c);
#pragma unroll
    for (int i = 0; i < kDistThreads / 64; ++i) sb += ws[i] * (double)exp2_from(wm[i], mf, d.c);
    st[split] = Stat{sb, mb, 0};
    if (a.first && split == 0)
      for (int i = a.splits; i < d.slots; ++i) st[i] = Stat{0, -__builtin_inff(), 0};
  }
}

// ---- the losses ----
// A row's sums joined. z_rest: of 2^((x - m) c) outside the list; z_list: of
// 2^((x - m_all) c) inside it, m_all >= m.
struct Whole {
  double z, log_z;   // of all columns, about m_all
  double rest_term;  // log z - log z_rest: -log of the mass outside the list
  double a, b;       // the gradient's factors (RowCoef)
};
__device__ __forceinline__ Whole whole(double z_rest, double z_list, float m, float m_all, double c,
                                       double mass, double rest) {
  Whole r;
  const double d = ((double)m - (double)m_all) * c;
  // nothing outside the list: m stands for no score
  r.z = z_list + (z_rest == 0 ? 0.0 : z_rest * exp2(d));
  r.log_z = log(r.z);
  r.rest_term = r.log_z - log(z_rest) - d * 0.693147180559945309417;
  r.a = mass / r.z;
  // with nothing outside the list b meets zeros alone: 0, or NaN where the row is
  r.b = z_rest == 0 ? (r.z - r.z) : r.a * exp2(d) - rest / z_rest;
  return r;
}

// the sum of L neighbouring lanes, in all of them
template <int L>
__device__ __forceinline__ double lanes_total(double v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, L);
  return v;
}
// L lanes a row. Bound by vector issue: three exponentials and two logarithms
// in 64 bits a row, whatever the lanes, and one a turn of the list.
template <int L>
__global__ __launch_bounds__(256) void distill_loss_kernel(DistillDev d, float *__restrict__ loss,
                                                           float *__restrict__ lse) {
  const int lane = threadIdx.x & (L - 1);
  const int64_t row = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (row >= d.n_rows) return;  // all lanes of a row
  const int32_t *sid = d.sid + row * d.k;
  const float *x = d.x + row * d.k, *p = d.p + row * d.k;
  const Stat *st = d.stat + row * d.slots;
  const RowTeach te = d.teach[row];
  // the columns outside the list by their own largest score: their mass, which the remaining
  // class divides by, must not vanish next to the list's
  float m = -__builtin_inff(), ml = -__builtin_inff();
  for (int i = lane; i < d.slots; i += L) m = fmaxf(m, st[i].m);
  for (int i = lane; i < d.k; i += L)
    if (sid[i] >= 0) ml = fmaxf(ml, x[i]);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor(m, o, L));
    ml = fmaxf(ml, __shfl_xor(ml, o, L));
  }
  const float mf = finite_max(m), ma = finite_max(fmaxf(m, ml));
  const double c = (double)d.c, ln2 = 0.693147180559945309417;
  double z_rest = 0, z_list = 0;
  for (int i = lane; i < d.slots; i += L) {
    const Stat s = st[i];
    if (s.s != 0) z_rest += s.s * exp2(((double)s.m - (double)mf) * c);
  }
  for (int i = lane; i < d.k; i += L)
    if (sid[i] >= 0) z_list += exp2(((double)x[i] - (double)ma) * c);
  z_rest = lanes_total<L>(z_rest);
  z_list = lanes_total<L>(z_list);
  const Whole z = whole(z_rest, z_list, mf, ma, c, te.mass, te.rest);
  double l = 0;
  for (int i = lane; i < d.k; i += L)
    if (sid[i] >= 0 && p[i] != 0)
      l += (double)p[i] * (z.log_z - ((double)x[i] - (double)ma) * c * ln2);
  l = lanes_total<L>(l) + te.entropy;
  if (te.rest != 0) l += te.rest * z.rest_term;
  const int32_t live = te.has && z.z != 0;  // a NaN is no 0
  if (lane == 0) {
    RowCoef r;
    r.a = z.a;
    r.b = z.b;
    r.m_all = ma;
    r.m = mf;
    r.live = live;
    r.pad = 0;
    d.coef[row] = r;
    loss[row] = live ? (float)l : 0.0f;
    if (lse) lse[row] = (float)((double)ma * c * ln2 + z.log_z);
  }
}

// ---- the gradient ----
struct GradArgs {
  DistillDev d;
  const void *x;
  void *g;
  const float *weights;  // nullable: 1
  int64_t ld, ldg, n_cols, col_begin, seg;
  int32_t splits;
};

template <typename T, typename G, int NT, int VPT>
__device__ __forceinline__ void store_tile(G *g, int64_t base, int64_t end, const float (&f)[VPT]) {
  constexpr int V = kVec<T>, W = kVec<G>;
#pragma unroll
  for (int v = 0; v < VPT / V; ++v) {
    const int64_t c = base + ((int64_t)v * NT + threadIdx.x) * V;
    if (c + V <= end) {
#pragma unroll
      for (int w = 0; w < V; w += W) {
        Vec<G> o;
#pragma unroll
        for (int e = 0; e < W; ++e) o.e[e] = from_f32<G>(f[v * V + w + e]);
        *reinterpret_cast<Vec<G> *>(g + c + w) = o;
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e < end) g[c + e] = from_f32<G>(f[v * V + e]);
    }
  }
}

// One pass, as a copy with an exponential: 10,000 x 8192 fp16 53 us, 6.2 TB/s.
template <typename T, typename G>
__global__ __launch_bounds__(kDistThreads) void distill_grad_kernel(GradArgs a) {
  const DistillDev &d = a.d;
  const int64_t row = blockIdx.x / (uint32_t)a.splits;
  const int32_t split = (int32_t)(blockIdx.x % (uint32_t)a.splits);
  const int64_t c0 = split * a.seg, c1 = c0 + a.seg < a.n_cols ? c0 + a.seg : a.n_cols;
  const T *x = static_cast<const T *>(a.x) + row * a.ld;
  G *g = static_cast<G *>(a.g) + row * a.ldg;
  const RowCoef r = d.coef[row];
  const double w = (a.weights ? (double)a.weights[row] : 1.0) * d.inv_tau;
  const float b = (float)(r.b * w);
  for (int64_t base = c0; base < c1; base += kDistTile) {
    float f[kDistVpt];
    load_tile<T, kDistThreads>(x, base, c1, f);
#pragma unroll
    for (int e = 0; e < kDistVpt; ++e) f[e] = r.live ? exp2_from(f[e], r.m, d.c) * b : 0.0f;
    store_tile<T, G, kDistThreads>(g, base, c1, f);
  }
  if (!r.live) return;  // uniform
  __syncthreads();      // the listed columns are written over what stands there
  for (int i = threadIdx.x; i < d.k; i += kDistThreads) {
    const int32_t id = d.sid[row * d.k + i];
    const int64_t o = (int64_t)id - a.col_begin;
    if (id >= 0 && o >= c0 && o < c1) {
      const double e = exp2(((double)d.x[row * d.k + i] - (double)r.m_all) * (double)d.c);
      g[o] = from_f32<G>((float)((e * r.a - (double)d.p[row * d.k + i]) * w));
    }
  }
}

// ---- whole rows in one launch ----
// One workgroup a row. A row that fits NT x VPT scores stays in registers from
// the load to the gradient: read once, written once, one exponential a score.
// A longer one is read a second time for the gradient, backwards, so that what
// was read last still comes from the caches. 4095 x 30522 bf16: 149 us, 3.4
// TB/s, bound by the chain of a row's life of which two run on a CU; 2000 x
// 100,000 fp32: 426 us, 3.8 TB/s of one reading and one writing.
struct RowsArgs {
  const void *x;
  void *g;  // nullable
  const int32_t *ids;
  const float *logits, *lse, *weights;
  float *loss;
  int64_t ld, ldg, n_cols;
  int32_t k;
  float c;
  double inv_tau;
};

template <int NT>
struct RowsShared {
  int32_t id[kDistMaxK];   // as given, -1 where unusable
  float x[kDistMaxK];      // the student's score of the entry
  double e[kDistMaxK];     // the entry's logit; then its mass before the common factor
  uint32_t bits[NT];  // the listed ones of a thread's scores
  double ws[6][16];
  float wf[3][16];
  double fa, fp;  // the factors of a listed score's exponential and of its entry's mass
  float b;        // of another score's exponential
  bool live;      // false: loss and gradient are 0
};

// The waves a SIMD holds: the other rows of a CU are what hides a row's chain
// of loads, barriers and reductions. Two workgroups of 1024 need 64 registers
// a thread: 20 values of 16-bit scores spill, 80 to 84 bytes of scratch a lane,
// and one workgroup without spills is slower all the same (220 against 149 us
// at 4095 x 30522). Smaller workgroups get the registers of a thread's scores
// (`regs`) and about 60 more, 2 to 4 values short of what 32 scores a thread
// take (12 to 20 bytes of scratch); 8 scores a thread spill nothing.
constexpr int rows_waves(int nt, int regs) {
  return nt == 1024 ? (regs <= 16 ? 8 : 4) : (regs <= 16 ? 6 : 5);
}

template <typename T, typename G, int NT, int VPT, bool LONG>
__global__ __launch_bounds__(NT, rows_waves(NT, VPT * (int)sizeof(T) / 4)) void distill_rows_kernel(
    RowsArgs a) {
  __shared__ RowsShared<NT> sh;
  constexpr int64_t kTileCols = (int64_t)NT * VPT;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(a.x) + row * a.ld;
  const int32_t *ids = a.ids + row * a.k;
  const float *logits = a.logits + row * a.k;
  RawTile<T, NT, VPT> f;
  if (!LONG) f.load(x, 0, a.n_cols);  // on its way while the list is worked on
  const double given = a.lse ? (double)a.lse[row] : 0.0;
  sh.bits[t] = 0;
#pragma unroll 1
  for (int i = t; i < a.k; i += NT) {
    const int32_t v = ids[i];
    const float l = logits[i];
    const bool ok = v >= 0 && v < a.n_cols && l != -__builtin_inff();
    sh.id[i] = ok ? v : -1;
    sh.x[i] = ok ? to_f32(x[v]) : -__builtin_inff();
    sh.e[i] = (double)l;
  }
  __syncthreads();
  // an entry takes part if no earlier one has its id; its column's bit is set
  uint32_t part = 0;  // of this thread's entries (k <= 1024: four at most)
  float mt = -__builtin_inff(), ml = -__builtin_inff(), m = -__builtin_inff();
#pragma unroll 1
  for (int i = t, j = 0; i < a.k; i += NT, ++j) {
    const int32_t v = sh.id[i];
    int dup = v < 0;
#pragma unroll 8
    for (int q = 0; q < i; ++q) dup |= sh.id[q] == v;
    if (!dup) {
      part |= 1u << j;
      mt = fmaxf(mt, (float)sh.e[i]);
      ml = fmaxf(ml, sh.x[i]);
      if (!LONG) {
        int word, bit;
        bit_of<T, NT>(v, word, bit);
        atomicOr(&sh.bits[word], 1u << bit);
      }
    }
  }
  __syncthreads();
  double z_rest = 0;
  if (LONG) {
    for (int64_t b0 = 0; b0 < a.n_cols; b0 += kTileCols) {
      for (int i = t, j = 0; i < a.k; i += NT, ++j) {
        const int64_t o = (int64_t)sh.id[i] - b0;
        if ((part >> j & 1u) && o >= 0 && o < kTileCols) {
          int word, bit;
          bit_of<T, NT>((int)o, word, bit);
          atomicOr(&sh.bits[word], 1u << bit);
        }
      }
      f.load(x, b0, a.n_cols);
      __syncthreads();
      const uint32_t listed = sh.bits[t];
      if (listed) {
        sh.bits[t] = 0;  // for the next tile: set behind the barrier below
#pragma unroll
        for (int e = 0; e < VPT; ++e)
          if (listed >> e & 1u) f.strike(e);
      }
      // a maximum of the thread's own; the workgroup's follows
      float mn = m;
#pragma unroll
      for (int e = 0; e < VPT; ++e) mn = fmaxf(mn, f.get(e));
      const float mf = finite_max(mn);
      float sum = 0;
#pragma unroll
      for (int e = 0; e < VPT; ++e) sum += exp2_from(f.get(e), mf, a.c);
      z_rest = z_rest * (double)exp2_from(m, mf, a.c) + (double)sum;
      m = mn;
      __syncthreads();
    }
  } else {
    const uint32_t listed = sh.bits[t];
    if (listed) {
#pragma unroll
      for (int e = 0; e < VPT; ++e)
        if (listed >> e & 1u) f.strike(e);
    }
#pragma unroll
    for (int e = 0; e < VPT; ++e) m = fmaxf(m, f.get(e));
  }
  const float mine = m;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor(m, o, 64));
    ml = fmaxf(ml, __shfl_xor(ml, o, 64));
    mt = fmaxf(mt, __shfl_xor(mt, o, 64));
  }
  if (lane == 0) {
    sh.wf[0][wave] = m;
    sh.wf[1][wave] = mt;
    sh.wf[2][wave] = ml;
  }
  __syncthreads();
  m = sh.wf[0][lane & (NT / 64 - 1)];
  mt = sh.wf[1][lane & (NT / 64 - 1)];
  ml = sh.wf[2][lane & (NT / 64 - 1)];
#pragma unroll
  for (int o = NT / 128; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor(m, o, 64));
    ml = fmaxf(ml, __shfl_xor(ml, o, 64));
    mt = fmaxf(mt, __shfl_xor(mt, o, 64));
  }
  const float mf = finite_max(m), ma = finite_max(fmaxf(m, ml));
  if (LONG) {
    z_rest *= (double)exp2_from(mine, mf, a.c);
  } else {
    f.forget();
    float sum = 0;
#pragma unroll
    for (int e = 0; e < VPT; ++e) sum += exp2_from(f.get(e), mf, a.c);
    z_rest = (double)sum;
    f.forget();
  }
  // sums: student's mass outside the list and inside; teacher's e, e log e and e (x - m), where
  // a listed entry's mass is e over their sum (or e itself); entries
  const double c = (double)a.c, ln2 = 0.693147180559945309417;
  {
    const double shift = a.lse ? given : (double)finite_max(mt) * a.inv_tau;
    double v[6] = {z_rest, 0, 0, 0, 0, 0};
#pragma unroll 1
    for (int i = t, j = 0; i < a.k; i += NT, ++j)
      if (part >> j & 1u) {
        const double d = ((double)sh.x[i] - (double)ma) * c;
        double s = exp2(d);
        asm volatile("" : "+v"(s));  // one function's temporaries at a time
        v[1] += s;
        const double y = sh.e[i] * a.inv_tau - shift, e = exp(y);
        v[2] += e;
        if (e != 0) {
          v[3] += e * y;
          v[4] += e * d;
        }
        v[5] += 1;
        sh.e[i] = e;
      }
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const double s = wave_total_f64(v[i]);
      if (lane == 63) sh.ws[i][wave] = s;
    }
  }
  __syncthreads();
  if (wave == 0) {
    double v[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = row16_sum(lane & 15, NT / 64, sh.ws[i]);
    const double scale = a.lse ? 1.0 : 1.0 / v[2];
    const double rest = !a.lse ? 0.0 : v[2] < 1 ? 1 - v[2] : v[2] >= 1 ? 0.0 : v[2];  // NaN stays
    // the list's mass: 1, or NaN where the logits are
    const double listed_mass = a.lse ? v[2] : 1.0 + (v[2] - v[2]);
    const Whole z = whole(v[0], v[1], mf, ma, c, listed_mass + rest, rest);
    const bool live = v[5] != 0 && z.z != 0;  // a NaN is no 0
    if (lane == 0) {
      // sum p log p, p = e scale; sum p (log z - (x - m)); the remaining class
      double l =
          v[3] * scale + (a.lse ? 0.0 : log(scale)) + listed_mass * z.log_z - v[4] * scale * ln2;
      if (rest != 0) l += rest * (log(rest) + z.rest_term);
      a.loss[row] = live ? (float)l : 0.0f;
      const double w = (a.weights ? (double)a.weights[row] : 1.0) * a.inv_tau;
      sh.fa = z.a * w;
      sh.fp = scale * w;
      sh.b = (float)(z.b * w);
      sh.live = live;
    }
  }
  if (!a.g) return;
  __syncthreads();
  const float b = sh.b;
  const bool live = sh.live;
  G *g = static_cast<G *>(a.g) + row * a.ldg;
  if (LONG) {  // backwards: the last tiles are still in the nearest cache
    for (int64_t b0 = (a.n_cols - 1) / kTileCols * kTileCols; b0 >= 0; b0 -= kTileCols) {
      f.load(x, b0, a.n_cols);
      f.store(g, b0, a.n_cols, live, mf, a.c, b);
    }
  } else {
    f.store(g, 0, a.n_cols, live, mf, a.c, b);
  }
  if (!live) return;  // uniform
  __syncthreads();    // the listed columns are written over what stands there
#pragma unroll 1
  for (int i = t, j = 0; i < a.k; i += NT, ++j)
    if (part >> j & 1u) {
      const double e = exp2(((double)sh.x[i] - (double)ma) * c);
      g[sh.id[i]] = from_f32<G>((float)(e * sh.fa - sh.e[i] * sh.fp));
    }
}

}  // namespace sps

struct sps_distill {
  sps::DistillDev d;
};

namespace {

using sps::DistillDev;
using sps::set_error;

// Whole rows go to one launch, a workgroup each, where a row fits a
// workgroup's registers (4 x 30,000: 11 us, in four launches 23) or where there
// are rows for half the card (128 x 200,000: 57 against 63 us); few long rows
// are cut among workgroups instead, in four launches (16 x 200,000: 20 us, in
// one 39; 64 x 200,000: 38 against 44).
constexpr int64_t kOneTile = 32768, kManyRows = 128;

constexpr int64_t kMax31 = 2147483647ll;

int32_t slots_of(int64_t n_rows) {
  if (n_rows <= 0 || n_rows >= sps::kDistFill) return 1;
  const int64_t s = (sps::kDistFill + n_rows - 1) / n_rows;
  return (int32_t)(s < sps::kMaxSlots ? s : sps::kMaxSlots);
}

// parts of a chunk's rows: as many as fill the card, none below a tile
void split_of(int64_t n_rows, int64_t n_cols, int32_t *splits, int64_t *seg) {
  int64_t s = slots_of(n_rows);
  const int64_t most = (n_cols + sps::kDistTile - 1) / sps::kDistTile;
  s = s < most ? s : most;
  s = s > 1 ? s : 1;
  int64_t g = ((n_cols + s - 1) / s + 7) / 8 * 8;
  if (g < 8) g = 8;
  s = (n_cols + g - 1) / g;
  *splits = (int32_t)(s > 1 ? s : 1);
  *seg = g;
}

struct Layout {
  size_t sid, p, x, teach, coef, stat, total;
};
Layout layout_of(int64_t n, int32_t k) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  Layout L;
  size_t at = 0;
  L.sid = at;
  at = up(at + (size_t)n * k * 4);
  L.p = at;
  at = up(at + (size_t)n * k * 4);
  L.x = at;
  at = up(at + (size_t)n * k * 4);
  L.teach = at;
  at = up(at + (size_t)n * sizeof(sps::RowTeach));
  L.coef = at;
  at = up(at + (size_t)n * sizeof(sps::RowCoef));
  L.stat = at;
  at = up(at + (size_t)n * slots_of(n) * sizeof(sps::Stat));
  L.total = at;
  return L;
}

sps_status check_sizes(int64_t n_rows, int32_t k, const char *what) {
  if (n_rows < 0) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: negative size", what);
  if (k < 1 || k > sps::kDistMaxK)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: k must be in [1, %d]", what, sps::kDistMaxK);
  if (n_rows >= kMax31) return set_error(SPS_ERR_OVERFLOW, "%s: rows must be below 2^31", what);
  // a workgroup a row at the most; more than one only of fewer than kDistFill rows
  return sps::check_grid(n_rows, 1024, what);
}

sps_status check_cols(int64_t n_cols, const char *what) {
  if (n_cols < 0) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: negative size", what);
  if (n_cols >= kMax31) return set_error(SPS_ERR_OVERFLOW, "%s: columns must be below 2^31", what);
  return SPS_OK;
}

bool one_launch(int64_t n_rows, int64_t n_cols) {
  return n_cols <= kOneTile || n_rows >= kManyRows;
}
// Whole rows in one launch keep nothing between kernels; the call still asks for an aligned
// workspace, the least there is.
size_t rows_bytes(int64_t n_rows, int64_t n_cols, int32_t k) {
  if (n_rows == 0) return 0;
  return one_launch(n_rows, n_cols) ? 256 : layout_of(n_rows, k).total;
}

// the checks of a list and its workspace of `need` bytes; fills d
sps_status make_dev(const int32_t *ids, const float *logits, int64_t n_rows, int32_t k,
                    int64_t n_cols, float tau, void *ws, size_t bytes, size_t need,
                    const char *what, DistillDev *d) {
  const sps_status st = check_cols(n_cols, what);
  if (st != SPS_OK) return st;
  if (!(tau >= 1e-6f && tau <= 1e6f))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: temperature must be in [1e-6, 1e6]", what);
  if (n_rows > 0 && (!ids || !logits))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL list", what);
  if (n_rows > 0 && !ws) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL workspace", what);
  if (bytes < need)
    return set_error(SPS_ERR_WORKSPACE_TOO_SMALL, "%s: need %zu bytes, got %zu", what, need, bytes);
  if (reinterpret_cast<uintptr_t>(ws) & 255)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", what);
  const Layout L = layout_of(n_rows, k);
  char *b = static_cast<char *>(ws);
  d->n_rows = n_rows;
  d->n_cols = n_cols;
  d->k = k;
  d->slots = slots_of(n_rows);
  d->c = (float)(1.44269504088896340736 / (double)tau);
  d->inv_tau = 1.0 / (double)tau;
  d->sid = reinterpret_cast<int32_t *>(b + L.sid);
  d->p = reinterpret_cast<float *>(b + L.p);
  d->x = reinterpret_cast<float *>(b + L.x);
  d->teach = reinterpret_cast<sps::RowTeach *>(b + L.teach);
  d->coef = reinterpret_cast<sps::RowCoef *>(b + L.coef);
  d->stat = reinterpret_cast<sps::Stat *>(b + L.stat);
  return SPS_OK;
}

// Lists of up to this are a wave's each, with little LDS and many at once
// (10,000 lists of 16: 10.6 us, by 256 threads 24; of 128: 21.6 against 35.8).
constexpr int kShortList = 128;

void launch_prepare(const DistillDev &d, const int32_t *ids, const float *logits, const float *lse,
                    hipStream_t s) {
  if (d.k <= kShortList)
    hipLaunchKernelGGL((sps::distill_prepare_kernel<64, kShortList>), dim3((uint32_t)d.n_rows), dim3(64), 0, s,
                       d, ids, logits, lse);
  else
    hipLaunchKernelGGL((sps::distill_prepare_kernel<256, sps::kDistMaxK>), dim3((uint32_t)d.n_rows), dim3(256), 0,
                       s, d, ids, logits, lse);
}

void launch_chunk(const DistillDev &d, const sps_scores *x, int32_t first, hipStream_t s) {
  sps::ChunkArgs a{};
  a.d = d;
  a.x = x->data;
  a.ld = x->ld;
  a.n_cols = x->n_cols;
  a.col_begin = x->col_begin;
  a.first = first != 0;
  split_of(d.n_rows, x->n_cols, &a.splits, &a.seg);
  const dim3 grid((uint32_t)(d.n_rows * a.splits)), block(sps::kDistThreads);
  if (x->dtype == SPS_F32)
    hipLaunchKernelGGL((sps::distill_chunk_kernel<float>), grid, block, 0, s, a);
  else if (x->dtype == SPS_F16)
    hipLaunchKernelGGL((sps::distill_chunk_kernel<sps::f16_t>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((sps::distill_chunk_kernel<sps::bf16_t>), grid, block, 0, s, a);
}

// 16 lanes a row where the rows fill the card, else a wave (full lists, no
// remaining class, whose two more logarithms and its term take 8.2 us at
// (10,000, 32)): (10,000, 32) 6.5 against 12.7 us, (10,000, 100) 11.4 : 14.0, (4000, 32) 5.1 : 7.0, (2000, 32)
// 5.0 : 5.5, (512, 8) 4.5 : 4.8, (50,000, 512) 183 : 195; but (4000, 100) 8.5 :
// 7.9, (512, 32) 5.0 : 4.7, (10,000, 512) 72 : 38. (Rows, list.)
constexpr int64_t kLossRows = 64;  // for each entry of the list
void launch_loss(const DistillDev &d, float *loss, float *lse, hipStream_t s) {
  const int64_t longest = d.k > d.slots ? d.k : d.slots;
  if (d.n_rows >= kLossRows * longest)
    hipLaunchKernelGGL((sps::distill_loss_kernel<16>), dim3((uint32_t)((d.n_rows + 15) / 16)),
                       dim3(256), 0, s, d, loss, lse);
  else
    hipLaunchKernelGGL((sps::distill_loss_kernel<64>), dim3((uint32_t)((d.n_rows + 3) / 4)),
                       dim3(256), 0, s, d, loss, lse);
}

sps_status check_grad(const sps_scores *x, const void *grad, int32_t dtype, int64_t ld,
                      const char *what) {
  if (dtype != x->dtype && dtype != SPS_F32)
    return set_error(SPS_ERR_INVALID_ARGUMENT,
                     "%s: the gradient's type is the scores' or float32", what);
  if (ld < x->n_cols)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: ld_grad below the columns", what);
  if (x->n_rows > 0 && (uint64_t)ld > (uint64_t)INT64_MAX / 4 / (uint64_t)x->n_rows)
    return set_error(SPS_ERR_OVERFLOW, "%s: n_rows * ld_grad overflows", what);
  if (x->n_rows > 0 && x->n_cols > 0 && !grad)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL gradient", what);
  if (reinterpret_cast<uintptr_t>(grad) % (uintptr_t)sps::dtype_size(dtype))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: gradient not aligned to its elements", what);
  if (x->n_rows > 0 && x->n_cols > 0) {
    // in place, or apart: a gradient that overlaps other scores would overwrite them unread
    const int64_t sx = sps::dtype_size(x->dtype), sg = sps::dtype_size(dtype);
    const bool same = x->data == grad && dtype == x->dtype && (ld == x->ld || x->n_rows == 1);
    if (!same && sps::rows_overlap({x->data, x->n_rows, x->n_cols * sx, x->ld * sx},
                                   {grad, x->n_rows, x->n_cols * sg, ld * sg}))
      return set_error(SPS_ERR_INVALID_ARGUMENT,
                       "%s: the gradient overlaps the scores without being them", what);
  }
  return SPS_OK;
}

void launch_grad(const DistillDev &d, const sps_scores *x, const float *weights, void *grad,
                 int32_t dtype, int64_t ldg, hipStream_t s) {
  if (x->n_cols == 0) return;
  sps::GradArgs a{};
  a.d = d;
  a.x = x->data;
  a.g = grad;
  a.weights = weights;
  a.ld = x->ld;
  a.ldg = ldg;
  a.n_cols = x->n_cols;
  a.col_begin = x->col_begin;
  split_of(d.n_rows, x->n_cols, &a.splits, &a.seg);
  const dim3 grid((uint32_t)(d.n_rows * a.splits)), block(sps::kDistThreads);
  using sps::bf16_t;
  using sps::f16_t;
  if (x->dtype == SPS_F32)
    hipLaunchKernelGGL((sps::distill_grad_kernel<float, float>), grid, block, 0, s, a);
  else if (x->dtype == SPS_F16 && dtype == SPS_F16)
    hipLaunchKernelGGL((sps::distill_grad_kernel<f16_t, f16_t>), grid, block, 0, s, a);
  else if (x->dtype == SPS_F16)
    hipLaunchKernelGGL((sps::distill_grad_kernel<f16_t, float>), grid, block, 0, s, a);
  else if (dtype == SPS_BF16)
    hipLaunchKernelGGL((sps::distill_grad_kernel<bf16_t, bf16_t>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((sps::distill_grad_kernel<bf16_t, float>), grid, block, 0, s, a);
}

template <typename T, typename G>
void launch_rows(const sps::RowsArgs &a, int64_t rows, hipStream_t s) {
  const dim3 grid((uint32_t)rows);
  if (a.n_cols <= 256 * 8)
    hipLaunchKernelGGL((sps::distill_rows_kernel<T, G, 256, 8, false>), grid, dim3(256), 0, s, a);
  else if (a.n_cols <= 256 * 32)
    hipLaunchKernelGGL((sps::distill_rows_kernel<T, G, 256, 32, false>), grid, dim3(256), 0, s, a);
  else if (a.n_cols <= 512 * 32)
    hipLaunchKernelGGL((sps::distill_rows_kernel<T, G, 512, 32, false>), grid, dim3(512), 0, s, a);
  else if (a.n_cols <= 1024 * 32)
    hipLaunchKernelGGL((sps::distill_rows_kernel<T, G, 1024, 32, false>), grid, dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL((sps::distill_rows_kernel<T, G, 1024, 32, true>), grid, dim3(1024), 0, s, a);
}

// a chunk of the batch's columns
sps_status check_chunk(const sps_distill *h, const sps_scores *x, const char *what) {
  if (!h) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL handle", what);
  const sps_status st = sps::check_scores(x, what);
  if (st != SPS_OK) return st;
  if (x->n_rows != h->d.n_rows)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: %lld rows of scores, %lld lists", what,
                     (long long)x->n_rows, (long long)h->d.n_rows);
  if (x->col_begin + x->n_cols > h->d.n_cols)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: columns past the batch's %lld", what,
                     (long long)h->d.n_cols);
  return SPS_OK;
}

}  // namespace

extern "C" {

sps_status sps_distill_workspace_size(int64_t n_rows, int32_t k, size_t *bytes) {
  if (!bytes) return set_error(SPS_ERR_INVALID_ARGUMENT, "NULL output pointer");
  const sps_status st = check_sizes(n_rows, k, "sps_distill_workspace_size");
  if (st != SPS_OK) return st;
  *bytes = layout_of(n_rows, k).total;
  return SPS_OK;
}

sps_status sps_distill_rows_workspace_size(int64_t n_rows, int64_t n_cols, int32_t k,
                                           size_t *bytes) {
  const char *what = "sps_distill_rows_workspace_size";
  if (!bytes) return set_error(SPS_ERR_INVALID_ARGUMENT, "NULL output pointer");
  sps_status st = check_sizes(n_rows, k, what);
  if (st == SPS_OK) st = check_cols(n_cols, what);
  if (st != SPS_OK) return st;
  *bytes = rows_bytes(n_rows, n_cols, k);
  return SPS_OK;
}

sps_status sps_distill_prepare(const int32_t *ids, const float *logits, const float *teacher_lse,
                               int64_t n_rows, int32_t k, int64_t n_cols, float temperature,
                               void *workspace, size_t workspace_bytes, void *stream,
                               sps_distill **out) {
  if (!out) return set_error(SPS_ERR_INVALID_ARGUMENT, "NULL output handle pointer");
  *out = nullptr;
  const char *what = "sps_distill_prepare";
  DistillDev d{};
  sps_status st = check_sizes(n_rows, k, what);
  if (st != SPS_OK) return st;
  st = make_dev(ids, logits, n_rows, k, n_cols, temperature, workspace, workspace_bytes,
                layout_of(n_rows, k).total, what, &d);
  if (st != SPS_OK) return st;
  sps_distill *h = new (std::nothrow) sps_distill;
  if (!h) return set_error(SPS_ERR_INVALID_ARGUMENT, "out of host memory");
  h->d = d;
  if (n_rows > 0) {
    launch_prepare(d, ids, logits, teacher_lse, reinterpret_cast<hipStream_t>(stream));
    st = sps::launch_status(what);
    if (st != SPS_OK) {
      delete h;
      return st;
    }
  }
  *out = h;
  return SPS_OK;
}

sps_status sps_distill_chunk(sps_distill *h, const sps_scores *scores, int32_t first,
                             void *stream) {
  const sps_status st = check_chunk(h, scores, "sps_distill_chunk");
  if (st != SPS_OK) return st;
  if (h->d.n_rows == 0) return SPS_OK;
  launch_chunk(h->d, scores, first, reinterpret_cast<hipStream_t>(stream));
  return sps::launch_status("sps_distill_chunk");
}

sps_status sps_distill_loss(sps_distill *h, float *loss, float *lse, void *stream) {
  if (!h) return set_error(SPS_ERR_INVALID_ARGUMENT, "sps_distill_loss: NULL handle");
  if (h->d.n_rows == 0) return SPS_OK;
  if (!loss) return set_error(SPS_ERR_INVALID_ARGUMENT, "sps_distill_loss: NULL output");
  launch_loss(h->d, loss, lse, reinterpret_cast<hipStream_t>(stream));
  return sps::launch_status("sps_distill_loss");
}

sps_status sps_distill_chunk_grad(sps_distill *h, const sps_scores *scores,
                                  const float *row_weights, void *grad, int32_t grad_dtype,
                                  int64_t ld_grad, void *stream) {
  sps_status st = check_chunk(h, scores, "sps_distill_chunk_grad");
  if (st == SPS_OK) st = check_grad(scores, grad, grad_dtype, ld_grad, "sps_distill_chunk_grad");
  if (st != SPS_OK) return st;
  if (h->d.n_rows == 0) return SPS_OK;
  launch_grad(h->d, scores, row_weights, grad, grad_dtype, ld_grad,
              reinterpret_cast<hipStream_t>(stream));
  return sps::launch_status("sps_distill_chunk_grad");
}

void sps_distill_destroy(sps_distill *h) { delete h; }

sps_status sps_distill_rows(const sps_scores *scores, const int32_t *ids, const float *logits,
                            const float *teacher_lse, int32_t k, float temperature,
                            const float *row_weights, float *loss, void *grad, int32_t grad_dtype,
                            int64_t ld_grad, void *workspace, size_t workspace_bytes,
                            void *stream) {
  const char *what = "sps_distill_rows";
  sps_status st = sps::check_scores(scores, what);
  if (st != SPS_OK) return st;
  if (scores->col_begin != 0)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: rows must be whole (col_begin 0)", what);
  DistillDev d{};
  st = check_sizes(scores->n_rows, k, what);
  if (st != SPS_OK) return st;
  st = make_dev(ids, logits, scores->n_rows, k, scores->n_cols, temperature, workspace,
                workspace_bytes, rows_bytes(scores->n_rows, scores->n_cols, k), what, &d);
  if (st != SPS_OK) return st;
  if (grad) st = check_grad(scores, grad, grad_dtype, ld_grad, what);
  if (st != SPS_OK) return st;
  if (d.n_rows == 0) return SPS_OK;
  if (!loss) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL loss", what);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (one_launch(scores->n_rows, scores->n_cols)) {
    sps::RowsArgs a{};
    a.x = scores->data;
    a.g = scores->n_cols > 0 ? grad : nullptr;
    a.ids = ids;
    a.logits = logits;
    a.lse = teacher_lse;
    a.weights = row_weights;
    a.loss = loss;
    a.ld = scores->ld;
    a.ldg = ld_grad;
    a.n_cols = scores->n_cols;
    a.k = k;
    a.c = d.c;
    a.inv_tau = d.inv_tau;
    using sps::bf16_t;
    using sps::f16_t;
    if (scores->dtype == SPS_F32) launch_rows<float, float>(a, d.n_rows, s);
    else if (scores->dtype == SPS_F16 && (grad_dtype == SPS_F16 || !grad))
      launch_rows<f16_t, f16_t>(a, d.n_rows, s);
    else if (scores->dtype == SPS_F16) launch_rows<f16_t, float>(a, d.n_rows, s);
    else if (grad_dtype == SPS_BF16 || !grad) launch_rows<bf16_t, bf16_t>(a, d.n_rows, s);
    else launch_rows<bf16_t, float>(a, d.n_rows, s);
    return sps::launch_status(what);
  }
  launch_prepare(d, ids, logits, teacher_lse, s);
  launch_chunk(d, scores, 1, s);
  launch_loss(d, loss, nullptr, s);
  if (grad) launch_grad(d, scores, row_weights, grad, grad_dtype, ld_grad, s);
  return sps::launch_status(what);
}

}  // extern "C"
