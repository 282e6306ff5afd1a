// sps_select.hip -- the best entries of rows of scores on gfx950: the running
// best k of every row over chunks of columns, the best k of (beam, column)
// over a group of rows, and the rows of states that follow their parents.
//
// Mathematics. A score x of row r has the key fl32(offset[r] + x); candidates
// are the keys above -inf (a NaN is none). With u the unsigned integer whose
// order is that of the key, the 64-bit integer (u << 32) | ~column is larger
// for the better candidate: by key, then by the lower column. All such
// integers of a row differ, so "the best k" is one set in one order, whatever
// the order in which workgroups, tiles or chunks reach it.
//
// What bounds it: reading the scores once. A workgroup holds a tile of a row
// in registers and the best k so far in LDS; after the first tile almost no
// element passes the k-th best, and the tile costs one compare an element.
// The first tile has no such bound yet: it takes a bound just below the k-th
// largest of its threads' own maxima, which at least k elements reach, so that
// little more than k elements are ever written to LDS and ranked.
#include "sps_rows.h"

namespace sps {

constexpr int kSelMaxK = 256;     // entries of a list: the public limit of k
constexpr int kSelThreads = 256;  // >= kSelMaxK: the threads' maxima bound the k-th best
constexpr int kSelBuf = 1024;     // candidates ranked at a time
constexpr int kBoundBits = 20;    // upper bits of a key that the first bound resolves
// Up to this k one maximum a thread bounds the k-th best, beyond two (8192 x
// 8192: k = 16 42.4 us with one, 44.0 with two; k = 96 56.9 and 56.7; k = 256
// 977, as the bound then is the least of 256 maxima, and 142).
constexpr int kOneMax = 96;
// a list that grows by 64-candidate steps must leave room for one
static_assert(kSelBuf >= 64 && kSelThreads >= kSelMaxK, "selection buffers");

struct SelShared {
  uint64_t buf[kSelBuf];
  uint64_t list[2][kSelMaxK];
  uint64_t best[kSelThreads];  // also 2 x kSelThreads upper halves
  // of three rounds: a wave may still read one round's while another pushes
  // the next one's, so the third is the one that can be cleared
  uint32_t cnt[3], full_at[3];
  uint32_t bound;
};

__device__ __forceinline__ uint64_t key_of(float f, uint32_t place) {
  const uint32_t u = order_bits(f);
  return u ? ((uint64_t)u << 32) | (uint32_t)~place : 0;
}

// k-th largest of the workgroup's `best` keys (0 where fewer than k of them
// are set), found bit by bit: every wave holds all keys and counts by ballot.
__device__ __forceinline__ uint64_t kth_of_best(const SelShared &sh, int k) {
  constexpr int N = kSelThreads / 64;
  const int lane = threadIdx.x & 63;
  uint32_t hi[N], lo[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t v = sh.best[i * 64 + lane];
    hi[i] = (uint32_t)(v >> 32);
    lo[i] = (uint32_t)v;
  }
  uint32_t th = 0;
  for (int b = 31; b >= 0; --b) {
    const uint32_t t = th | (1u << b);
    int c = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) c += __popcll(__ballot(hi[i] >= t));
    if (c >= k) th = t;
  }
  if (th == 0) return 0;
  // of the keys with this upper half, the (k - above)-th largest
  int above = 0, same = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    above += __popcll(__ballot(hi[i] > th));
    same += __popcll(__ballot(hi[i] == th));
  }
  uint32_t tl = 0;
  if (above + same > k) {
    for (int b = 31; b >= 0; --b) {
      const uint32_t t = tl | (1u << b);
      int c = above;
#pragma unroll
      for (int i = 0; i < N; ++i) c += __popcll(__ballot(hi[i] == th && lo[i] >= t));
      if (c >= k) tl = t;
    }
  }
  return ((uint64_t)th << 32) | tl;
}

// The largest multiple of 2^(32 - kBoundBits) that at least k of N x 64 keys'
// upper halves reach (0 where fewer than k are set), by one wave.
template <int N>
__device__ __forceinline__ uint32_t kth_bound(const uint32_t *best, int k) {
  const int lane = threadIdx.x & 63;
  uint32_t h[N];
#pragma unroll
  for (int i = 0; i < N; ++i) h[i] = best[i * 64 + lane];
  uint32_t th = 0;
  for (int b = 31; b >= 32 - kBoundBits; --b) {
    const uint32_t t = th | (1u << b);
    int c = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) c += __popcll(__ballot(h[i] >= t));
    if (c >= k) th = t;
  }
  return th;
}

// Puts the m candidates of `buf` into the sorted list (n of at most k): a
// key's place is the number of larger keys. Every key is compared with the m
// new ones, a new one with the list by bisection; a column offered again with
// the same score has its listed key once more and stands behind it. Returns
// the list's length; the list is then list[1 - cur].
__device__ __forceinline__ int merge_buf(SelShared &sh, int cur, int n, int m, int k) {
  const uint64_t *list = sh.list[cur];
  uint64_t *to = sh.list[1 - cur];
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const uint64_t v = list[i];
    int r = i;
#pragma unroll 8
    for (int j = 0; j < m; ++j) r += sh.buf[j] > v;
    if (r < k) to[r] = v;
  }
  for (int i = threadIdx.x; i < m; i += kSelThreads) {
    const uint64_t v = sh.buf[i];
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (list[mid] >= v) lo = mid + 1;
      else hi = mid;
    }
    int r = lo;
#pragma unroll 8
    for (int j = 0; j < m; ++j) r += sh.buf[j] > v;
    if (r < k) to[r] = v;
  }
  return n + m < k ? n + m : k;
}

// One tile: thread t offers keys f[i] (-inf or NaN for none). key(i) gives the
// 64-bit integer of the thread's i-th element, with places ascending in i; it
// loads the element once more, which the few candidates of a tile are cheaper
// with than every element with an integer key of its own. Updates the list
// list[cur][0, n); all threads must call it. `rnd` is the round (0, 1, 2, 0,
// ...), the same in all threads.
template <int VPT, typename Key>
__device__ __forceinline__ void offer_tile(SelShared &sh, const float (&f)[VPT], Key key, int k,
                                           int &cur, int &n, int &rnd) {
  static_assert(VPT <= 32, "one bit an element");
  const int t = threadIdx.x, lane = t & 63;
  float m0 = -__builtin_inff(), m1 = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < VPT / 2; ++i) {
    m0 = fmaxf(m0, f[i]);
    m1 = fmaxf(m1, f[VPT / 2 + i]);
  }
  uint64_t thr = 0;  // candidates are above it
  float tf = -3.4028234663852886e38f;  // none is below it: every key above -inf so far
  if (n < k) {  // no k-th best yet: bound it by the threads' maxima
    uint32_t *best = reinterpret_cast<uint32_t *>(sh.best);
    if (k <= kOneMax) {
      best[t] = order_bits(fmaxf(m0, m1));
    } else {
      best[2 * t] = order_bits(m0);
      best[2 * t + 1] = order_bits(m1);
    }
    __syncthreads();
    if (t < 64) {
      const uint32_t b = k <= kOneMax ? kth_bound<kSelThreads / 64>(best, k)
                                      : kth_bound<2 * kSelThreads / 64>(best, k);
      if (t == 0) sh.bound = b;
    }
    __syncthreads();
    if (sh.bound) {
      tf = unorder_bits(sh.bound);
      thr = ((uint64_t)sh.bound << 32) - 1;
    }
  } else {
    thr = sh.list[cur][k - 1];
    tf = unorder_bits((uint32_t)(thr >> 32));
  }
  uint32_t pend = 0;  // element i in bit VPT - 1 - i
  if (__ballot(fmaxf(m0, m1) >= tf)) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      pend = pend << 1 | (f[i] >= tf ? 1u : 0u);
      if (i % 4 == 3) asm volatile("" : "+v"(pend));  // not all terms first
    }
  }
  for (;;) {
    // candidates into the buffer, one of each lane at a time, while they fit
    bool full = false;
    while (!full && __ballot(pend != 0)) {
      const int bit = 31 - __builtin_clz(pend | 1u);
      const uint64_t v = pend ? key(VPT - 1 - bit) : 0;
      const bool c = v > thr;
      const uint64_t mask = __ballot(c);
      uint32_t at = 0;
      if (mask != 0) {
        if (lane == 0) at = atomicAdd(&sh.cnt[rnd], (uint32_t)__popcll(mask));
        at = __builtin_amdgcn_readfirstlane(at);
        if (at + (uint32_t)__popcll(mask) > (uint32_t)kSelBuf) {
          // every later request fails too: places only grow
          if (lane == 0) atomicMin(&sh.full_at[rnd], at);
          full = true;
        } else if (c) {
          sh.buf[at + (uint32_t)__popcll(mask & ((1ull << lane) - 1))] = v;
        }
      }
      if (!full) pend &= ~(1u << bit);
    }
    __syncthreads();
    const uint32_t cnt = sh.cnt[rnd], full_at = sh.full_at[rnd];
    rnd = rnd == 2 ? 0 : rnd + 1;
    if (t == 0) {  // the round after the next: read before the barrier above
      const int later = rnd == 2 ? 0 : rnd + 1;
      sh.cnt[later] = 0;
      sh.full_at[later] = ~0u;
    }
    if (cnt == 0) return;
    const int m = (int)(cnt < full_at ? cnt : full_at);
    const int n2 = merge_buf(sh, cur, n, m, k);
    __syncthreads();
    cur ^= 1;
    n = n2;
    if (full_at == ~0u) return;
    // what did not fit, as with many equal keys: bounded by the list's k-th best and by the
    // k-th largest of the threads' best, now to the last bit
    thr = n < k ? 0 : sh.list[cur][k - 1];
    uint64_t mx = 0;
    uint32_t left = 0;
    while (pend) {
      const int bit = 31 - __builtin_clz(pend);
      pend &= ~(1u << bit);
      const uint64_t v = key(VPT - 1 - bit);
      if (v > thr) left |= 1u << bit;
      if (v > thr && v > mx) mx = v;
    }
    pend = left;
    sh.best[t] = mx;
    __syncthreads();
    const uint64_t b = kth_of_best(sh, k);
    if (b > thr) thr = b - 1;
  }
}

__device__ __forceinline__ void sel_init(SelShared &sh) {
  if (threadIdx.x < 3) {
    sh.cnt[threadIdx.x] = 0;
    sh.full_at[threadIdx.x] = ~0u;
  }
}

struct SelArgs {
  const void *x;
  int64_t ld, n_cols, col_begin;
  const float *offsets;  // nullable
  int32_t k, splits;
  int64_t seg;           // columns of a split
  int32_t first;         // the lists hold nothing yet
  float *top_scores;     // [rows][k], splits == 1
  int32_t *top_cols;
  uint64_t *parts;       // [rows][splits][k], splits > 1 (or the beam path)
};

// Best k of columns [split * seg, ...) of one row. With parts, they are
// written there as keys (0 behind the last); without, they join the row's list.
// Tiles of 256 threads x 32 scores: with 16 a thread the first chunk's lists
// are merged twice as often (808 against 696 us for two chunks of 50,000 x
// 8192), and 72 registers leave six workgroups a CU. Reads at 4.8 TB/s there
// (k = 100, the lists' growth included) and at 5.2 TB/s from 80 rows of 2M.
template <typename T, int VPT>
__global__ __launch_bounds__(kSelThreads, 6) void select_kernel(SelArgs a) {
  __shared__ SelShared sh;
  constexpr int V = kVec<T>, NV = VPT / V;
  const int64_t row = blockIdx.x / (uint32_t)a.splits;
  const int32_t split = (int32_t)(blockIdx.x % (uint32_t)a.splits);
  const int64_t c0 = split * a.seg;
  const int64_t c1 = c0 + a.seg < a.n_cols ? c0 + a.seg : a.n_cols;
  const T *x = static_cast<const T *>(a.x) + row * a.ld;
  const float off = a.offsets ? a.offsets[row] : 0.0f;
  const int t = threadIdx.x;
  int cur = 0, n = 0, rnd = 0;
  sel_init(sh);
  if (!a.parts && !a.first) {
    int ok = 0;
    if (t < a.k) {
      const float s = a.top_scores[row * a.k + t];
      const int32_t c = a.top_cols[row * a.k + t];
      const uint32_t o = order_bits(s);
      ok = c >= 0 && o != 0;
      sh.list[0][t] = ok ? ((uint64_t)o << 32) | (uint32_t)~(uint32_t)c : 0;
    }
    n = __syncthreads_count(ok);  // filled places come first
  }
  __syncthreads();
  for (int64_t base = c0; base < c1; base += kSelThreads * VPT) {
    float f[VPT];
    if (base + kSelThreads * VPT <= c1) {  // a whole tile: all loads in flight
      Vec<T> w[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v)
        w[v] = *reinterpret_cast<const Vec<T> *>(x + base + ((int64_t)v * kSelThreads + t) * V);
#pragma unroll
      for (int i = 0; i < VPT; ++i) f[i] = to_f32(w[i / V].e[i % V]) + off;
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t c = base + ((int64_t)v * kSelThreads + t) * V;
        if (c + V <= c1) {
          const Vec<T> w = *reinterpret_cast<const Vec<T> *>(x + c);
#pragma unroll
          for (int e = 0; e < V; ++e) f[v * V + e] = to_f32(w.e[e]) + off;
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e)
            f[v * V + e] = c + e < c1 ? to_f32(x[c + e]) + off : -__builtin_inff();
        }
      }
    }
    offer_tile<VPT>(
        sh, f,
        [&](int i) {
          const int64_t c = base + ((int64_t)(i / V) * kSelThreads + t) * V + i % V;
          return c < c1 ? key_of(to_f32(x[c]) + off, (uint32_t)(a.col_begin + c)) : (uint64_t)0;
        },
        a.k, cur, n, rnd);
  }
  if (t < a.k) {
    const uint64_t v = t < n ? sh.list[cur][t] : 0;
    if (a.parts) {
      a.parts[(row * a.splits + split) * a.k + t] = v;
    } else {
      a.top_scores[row * a.k + t] = v ? unorder_bits((uint32_t)(v >> 32)) : -__builtin_inff();
      a.top_cols[row * a.k + t] = v ? (int32_t)~(uint32_t)v : -1;
    }
  }
}

// The lists of a row's splits joined with the row's running list.
struct FoldArgs {
  const uint64_t *parts;
  int32_t lists, k, first;
  float *top_scores;
  int32_t *top_cols;
};

constexpr int kJoinVpt = 8;

__global__ __launch_bounds__(kSelThreads) void select_fold_kernel(FoldArgs a) {
  __shared__ SelShared sh;
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x;
  int cur = 0, n = 0, rnd = 0;
  sel_init(sh);
  if (!a.first) {
    int ok = 0;
    if (t < a.k) {
      const uint32_t o = order_bits(a.top_scores[row * a.k + t]);
      const int32_t c = a.top_cols[row * a.k + t];
      ok = c >= 0 && o != 0;
      sh.list[0][t] = ok ? ((uint64_t)o << 32) | (uint32_t)~(uint32_t)c : 0;
    }
    n = __syncthreads_count(ok);
  }
  __syncthreads();
  const int64_t total = (int64_t)a.lists * a.k;
  const uint64_t *p = a.parts + row * total;
  for (int64_t base = 0; base < total; base += kSelThreads * kJoinVpt) {
    float f[kJoinVpt];
#pragma unroll
    for (int i = 0; i < kJoinVpt; ++i) {
      const int64_t at = base + (int64_t)i * kSelThreads + t;
      const uint64_t v = at < total ? p[at] : 0;
      f[i] = v ? unorder_bits((uint32_t)(v >> 32)) : -__builtin_inff();
    }
    offer_tile<kJoinVpt>(
        sh, f,
        [&](int i) {
          const int64_t at = base + (int64_t)i * kSelThreads + t;
          return at < total ? p[at] : (uint64_t)0;
        },
        a.k, cur, n, rnd);
  }
  if (t < a.k) {
    const uint64_t v = t < n ? sh.list[cur][t] : 0;
    a.top_scores[row * a.k + t] = v ? unorder_bits((uint32_t)(v >> 32)) : -__builtin_inff();
    a.top_cols[row * a.k + t] = v ? (int32_t)~(uint32_t)v : -1;
  }
}

// Best k of a group's lists: beams x splits lists of k_in, sorted, beams
// first, a beam's splits by ascending columns. Among equal keys a place in
// this order stands for (beam, column): lists of one beam hold ascending
// column ranges, and a list has its equal keys by ascending column.
struct JoinArgs {
  const uint64_t *parts;   // keys, or
  const float *in_scores;  // scores and columns of running lists
  const int32_t *in_cols;
  int32_t beams, splits, k_in, k;
  float *scores;
  int32_t *parents, *cols;
};

__global__ __launch_bounds__(kSelThreads) void beam_join_kernel(JoinArgs a) {
  __shared__ SelShared sh;
  const int64_t group = blockIdx.x;
  const int t = threadIdx.x;
  const int64_t per_beam = (int64_t)a.splits * a.k_in, total = per_beam * a.beams;
  const int64_t at0 = group * total;
  int cur = 0, n = 0, rnd = 0;
  sel_init(sh);
  __syncthreads();
  for (int64_t base = 0; base < total; base += kSelThreads * kJoinVpt) {
    float f[kJoinVpt];
#pragma unroll
    for (int i = 0; i < kJoinVpt; ++i) {
      const int64_t at = base + (int64_t)i * kSelThreads + t;
      f[i] = -__builtin_inff();
      if (at < total) {
        if (a.parts) {
          const uint32_t u = (uint32_t)(a.parts[at0 + at] >> 32);
          if (u) f[i] = unorder_bits(u);
        } else if (a.in_cols[at0 + at] >= 0) {
          f[i] = a.in_scores[at0 + at];
        }
      }
    }
    offer_tile<kJoinVpt>(
        sh, f,
        [&](int i) {
          const int64_t at = base + (int64_t)i * kSelThreads + t;
          if (at >= total || (!a.parts && a.in_cols[at0 + at] < 0)) return (uint64_t)0;
          const float x = a.parts ? unorder_bits((uint32_t)(a.parts[at0 + at] >> 32))
                                  : a.in_scores[at0 + at];
          return key_of(x, (uint32_t)at);
        },
        a.k, cur, n, rnd);
  }
  if (t < a.k) {
    const uint64_t v = t < n ? sh.list[cur][t] : 0;
    const int64_t o = group * a.k + t;
    int32_t parent = -1, col = -1;
    float s = -__builtin_inff();
    if (v) {
      const int64_t at = (int64_t)(uint32_t)~(uint32_t)v;
      s = unorder_bits((uint32_t)(v >> 32));
      parent = (int32_t)(group * a.beams + at / per_beam);
      col = a.parts ? (int32_t)~(uint32_t)a.parts[at0 + at] : a.in_cols[at0 + at];
    }
    a.scores[o] = s;
    a.parents[o] = parent;
    a.cols[o] = col;
  }
}

// A whole group by one workgroup: its beams' rows as one run of places b *
// n_cols + column. For the small groups of a latency-bound step, where a
// second launch would cost more than the scores.
struct GroupArgs {
  const void *x;
  int64_t ld, n_cols, col_begin;
  const float *offsets;  // nullable
  int32_t beams, k;
  float *scores;
  int32_t *parents, *cols;
};

template <typename T, int VPT>
__global__ __launch_bounds__(kSelThreads) void beam_group_kernel(GroupArgs a) {
  __shared__ SelShared sh;
  constexpr int V = kVec<T>, NV = VPT / V;
  const int t = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * a.beams;
  const T *x = static_cast<const T *>(a.x) + row0 * a.ld;
  const float *off = a.offsets ? a.offsets + row0 : nullptr;
  const uint32_t cols = (uint32_t)a.n_cols, total = cols * (uint32_t)a.beams;  // below 2^32
  auto at = [&](uint32_t p) {
    const uint32_t b = p / cols;
    return to_f32(x[b * a.ld + (p - b * cols)]) + (off ? off[b] : 0.0f);
  };
  int cur = 0, n = 0, rnd = 0;
  sel_init(sh);
  __syncthreads();
  for (uint32_t base = 0; base < total; base += kSelThreads * VPT) {
    float f[VPT];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint32_t p = base + (uint32_t)(v * kSelThreads + t) * V;
      const uint32_t b = p < total ? p / cols : 0, c = p - b * cols;
      if (p + V <= total && c + V <= cols) {
        const Vec<T> w = *reinterpret_cast<const Vec<T> *>(x + b * a.ld + c);
        const float o = off ? off[b] : 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) f[v * V + e] = to_f32(w.e[e]) + o;
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[v * V + e] = p + e < total ? at(p + e) : -__builtin_inff();
      }
    }
    offer_tile<VPT>(
        sh, f,
        [&](int i) {
          const uint32_t p = base + (uint32_t)(i / V * kSelThreads + t) * V + (uint32_t)(i % V);
          return p < total ? key_of(at(p), p) : (uint64_t)0;
        },
        a.k, cur, n, rnd);
  }
  if (t < a.k) {
    const uint64_t v = t < n ? sh.list[cur][t] : 0;
    const int64_t o = (int64_t)blockIdx.x * a.k + t;
    const uint32_t p = ~(uint32_t)v, b = v ? p / cols : 0;
    a.scores[o] = v ? unorder_bits((uint32_t)(v >> 32)) : -__builtin_inff();
    a.parents[o] = v ? (int32_t)(row0 + b) : -1;
    a.cols[o] = v ? (int32_t)(a.col_begin + (p - b * cols)) : -1;
  }
}

// ---- states ----
constexpr int kMaxStates = 8;      // states of one launch
constexpr int kPieceBytes = 16384; // of a row, copied by one workgroup

struct StateArgs {
  const uint8_t *src[kMaxStates];
  uint8_t *dst[kMaxStates];
  int64_t bytes[kMaxStates], src_stride[kMaxStates], dst_stride[kMaxStates];
  int32_t pieces[kMaxStates];  // of a row
  int64_t first[kMaxStates + 1];
  int32_t width[kMaxStates];   // 16, 4 or 1: the widest that rows and strides are multiples of
  int32_t n;
  const int32_t *parents;
  int64_t n_rows;
};

template <typename W>
__device__ __forceinline__ void copy_piece(const uint8_t *src, uint8_t *dst, int64_t n) {
  const int64_t m = n / (int64_t)sizeof(W);
  const W *s = reinterpret_cast<const W *>(src);
  W *d = reinterpret_cast<W *>(dst);
  for (int64_t i = threadIdx.x; i < m; i += 256) d[i] = src ? s[i] : W{};
}

// A piece of a row a workgroup: 256 rows of 64 KB move at 4.9 TB/s (7 us).
__global__ __launch_bounds__(256) void reorder_kernel(StateArgs a) {
  const int64_t b = blockIdx.x;
  int i = 0;
  while (i + 1 < a.n && b >= a.first[i + 1]) ++i;
  const int64_t q = b - a.first[i];
  const int64_t row = q / a.pieces[i], o = (q % a.pieces[i]) * kPieceBytes;
  const int64_t n = a.bytes[i] - o < kPieceBytes ? a.bytes[i] - o : kPieceBytes;
  const int32_t p = a.parents[row];
  const bool there = p >= 0 && p < a.n_rows;
  const uint8_t *src = there ? a.src[i] + p * a.src_stride[i] + o : nullptr;
  uint8_t *dst = a.dst[i] + row * a.dst_stride[i] + o;
  if (a.width[i] == 16) copy_piece<uint4>(src, dst, n);
  else if (a.width[i] == 4) copy_piece<uint32_t>(src, dst, n);
  else copy_piece<uint8_t>(src, dst, n);
}

}  // namespace sps

namespace {

constexpr int64_t kMax31 = 2147483647ll;
constexpr int64_t kMaxPieces = 4294967295ll / 256;  // pieces of states in a launch

// Workgroups that fill the card, and the fewest columns worth one of them (2 x
// 100,000 scores: 10.4 us, with 4096 columns 10.9, with 16384 12.7; 128 x
// 32768: 10.4, 11.7, 13.2).
constexpr int64_t kFill = 1024, kMinSeg = 8192;

struct Split {
  int32_t splits;
  int64_t seg;
};
Split split_of(int64_t n_rows, int64_t n_cols) {
  int64_t s = 1;
  if (n_rows > 0 && n_rows < kFill) {
    const int64_t least = (kFill + n_rows - 1) / n_rows, most = (n_cols + kMinSeg - 1) / kMinSeg;
    s = least < most ? least : most > 1 ? most : 1;
    if (s == least) {  // of up to half as many again, the one that leaves the last round fullest
      double best = 0;
      for (int64_t c = least; c <= least + least / 2 && c <= most; ++c) {
        const double part = (double)(n_rows * c), fill = part / (double)((n_rows * c + 255) / 256 * 256);
        if (fill > best + 0.02) {
          best = fill;
          s = c;
        }
      }
    }
  }
  int64_t seg = (n_cols + s - 1) / s;
  seg = (seg + 7) / 8 * 8;  // whole vectors
  if (seg < 8) seg = 8;
  s = (n_cols + seg - 1) / seg;
  return {(int32_t)(s > 1 ? s : 1), seg};
}

// Groups of up to this many scores go to one workgroup each, in one launch (4
// beams of 512 columns: 4.6 us, in two launches 8.7; of 4096: 9.8 both ways,
// 512 such groups 11.7 against 16.8; of 8192: 16.8 against 9.1).
constexpr int64_t kOneGroup = 16384;
bool one_launch(int64_t n_cols, int32_t beams) { return n_cols <= kOneGroup / beams; }

template <typename T>
void launch_group(const sps::GroupArgs &a, int64_t groups, hipStream_t s) {
  const dim3 grid((uint32_t)groups), block(sps::kSelThreads);
  if (a.n_cols * a.beams <= sps::kSelThreads * 8)
    hipLaunchKernelGGL((sps::beam_group_kernel<T, 8>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((sps::beam_group_kernel<T, 32>), grid, block, 0, s, a);
}

// Short segments take tiles of 8 scores a thread (4096 x 2048 scores: 11.8 us,
// with 32 a thread 17.9).
template <typename T>
void launch_select(const sps::SelArgs &a, int64_t rows, hipStream_t s) {
  const uint32_t grid = (uint32_t)(rows * a.splits);
  if (a.seg <= sps::kSelThreads * 8)
    hipLaunchKernelGGL((sps::select_kernel<T, 8>), dim3(grid), dim3(sps::kSelThreads), 0, s, a);
  else
    hipLaunchKernelGGL((sps::select_kernel<T, 32>), dim3(grid), dim3(sps::kSelThreads), 0, s, a);
}

void launch_select(int32_t dtype, const sps::SelArgs &a, int64_t rows, hipStream_t s) {
  if (dtype == SPS_F32) launch_select<float>(a, rows, s);
  else if (dtype == SPS_F16) launch_select<sps::f16_t>(a, rows, s);
  else launch_select<sps::bf16_t>(a, rows, s);
}

sps_status check_k(int32_t k, const char *what) {
  if (k < 1 || k > sps::kSelMaxK)
    return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "%s: k must be in [1, %d]", what,
                          sps::kSelMaxK);
  return SPS_OK;
}

size_t parts_bytes(int64_t n_rows, const Split &sp, int32_t k) {
  return (size_t)n_rows * (size_t)sp.splits * (size_t)k * 8;
}

sps_status check_ws(const void *ws, size_t have, size_t need, const char *what) {
  if (need == 0) return SPS_OK;
  if (!ws) return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL workspace", what);
  if (have < need)
    return sps::set_error(SPS_ERR_WORKSPACE_TOO_SMALL, "%s: need %zu bytes, got %zu", what, need,
                          have);
  if (reinterpret_cast<uintptr_t>(ws) & 15)
    return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "%s: workspace must be 16-byte aligned", what);
  return SPS_OK;
}

}  // namespace

extern "C" {

sps_status sps_select_workspace_size(int64_t n_rows, int64_t n_cols, int32_t k, size_t *bytes) {
  if (!bytes) return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "NULL output pointer");
  if (n_rows < 0 || n_cols < 0)
    return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "negative size");
  if (n_rows >= kMax31 || n_cols >= kMax31)
    return sps::set_error(SPS_ERR_OVERFLOW, "sizes must be below 2^31");
  const sps_status st = check_k(k, "sps_select_workspace_size");
  if (st != SPS_OK) return st;
  const Split sp = split_of(n_rows, n_cols);
  *bytes = sp.splits > 1 ? parts_bytes(n_rows, sp, k) : 0;
  return SPS_OK;
}

sps_status sps_select_chunk(const sps_scores *scores, const float *offsets, int32_t k,
                            int32_t first, float *top_scores, int32_t *top_cols, void *workspace,
                            size_t workspace_bytes, void *stream) {
  sps_status st = sps::check_scores(scores, "sps_select_chunk");
  if (st != SPS_OK) return st;
  st = check_k(k, "sps_select_chunk");
  if (st != SPS_OK) return st;
  const int64_t rows = scores->n_rows;
  if (rows == 0) return SPS_OK;
  if (!top_scores || !top_cols)
    return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "sps_select_chunk: NULL lists");
  const Split sp = split_of(rows, scores->n_cols);
  const size_t need = sp.splits > 1 ? parts_bytes(rows, sp, k) : 0;
  st = check_ws(workspace, workspace_bytes, need, "sps_select_chunk");
  if (st != SPS_OK) return st;
  st = sps::check_grid(rows * sp.splits, sps::kSelThreads, "sps_select_chunk");
  if (st != SPS_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  sps::SelArgs a{};
  a.x = scores->data;
  a.ld = scores->ld;
  a.n_cols = scores->n_cols;
  a.col_begin = scores->col_begin;
  a.offsets = offsets;
  a.k = k;
  a.splits = sp.splits;
  a.seg = sp.seg;
  a.first = first != 0;
  a.top_scores = top_scores;
  a.top_cols = top_cols;
  a.parts = sp.splits > 1 ? static_cast<uint64_t *>(workspace) : nullptr;
  launch_select(scores->dtype, a, rows, s);
  if (sp.splits > 1) {
    sps::FoldArgs f{a.parts, sp.splits, k, first != 0, top_scores, top_cols};
    hipLaunchKernelGGL(sps::select_fold_kernel, dim3((uint32_t)rows), dim3(sps::kSelThreads), 0, s,
                       f);
  }
  return sps::launch_status("sps_select_chunk");
}

static sps_status check_beams(int64_t n_rows, int32_t beams, int64_t lists, int32_t k_in,
                              const char *what) {
  if (beams < 1 || n_rows % beams)
    return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "%s: %lld rows are no groups of %d beams",
                          what, (long long)n_rows, beams);
  if ((int64_t)beams * lists > kMax31 / k_in)
    return sps::set_error(SPS_ERR_OVERFLOW, "%s: beams x lists x k reaches 2^31", what);
  return SPS_OK;
}

sps_status sps_beam_workspace_size(int64_t n_rows, int64_t n_cols, int32_t beams, int32_t k,
                                   size_t *bytes) {
  size_t unused = 0;
  sps_status st = sps_select_workspace_size(n_rows, n_cols, k, &unused);
  if (st != SPS_OK) return st;
  if (!bytes) return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "NULL output pointer");
  const Split sp = split_of(n_rows, n_cols);
  st = check_beams(n_rows, beams, sp.splits, k, "sps_beam_workspace_size");
  if (st != SPS_OK) return st;
  *bytes = one_launch(n_cols, beams) ? 0 : parts_bytes(n_rows, sp, k);
  return SPS_OK;
}

sps_status sps_beam_select(const sps_scores *scores, const float *beam_scores, int32_t beams,
                           int32_t k, float *out_scores, int32_t *out_parents, int32_t *out_cols,
                           void *workspace, size_t workspace_bytes, void *stream) {
  sps_status st = sps::check_scores(scores, "sps_beam_select");
  if (st != SPS_OK) return st;
  st = check_k(k, "sps_beam_select");
  if (st != SPS_OK) return st;
  const int64_t rows = scores->n_rows;
  const Split sp = split_of(rows, scores->n_cols);
  st = check_beams(rows, beams, sp.splits, k, "sps_beam_select");
  if (st != SPS_OK) return st;
  if (rows == 0) return SPS_OK;
  if (!out_scores || !out_parents || !out_cols)
    return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "sps_beam_select: NULL output");
  st = sps::check_grid(rows * sp.splits, sps::kSelThreads, "sps_beam_select");
  if (st != SPS_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (one_launch(scores->n_cols, beams)) {
    sps::GroupArgs g{};
    g.x = scores->data;
    g.ld = scores->ld;
    g.n_cols = scores->n_cols;
    g.col_begin = scores->col_begin;
    g.offsets = beam_scores;
    g.beams = beams;
    g.k = k;
    g.scores = out_scores;
    g.parents = out_parents;
    g.cols = out_cols;
    if (scores->dtype == SPS_F32) launch_group<float>(g, rows / beams, s);
    else if (scores->dtype == SPS_F16) launch_group<sps::f16_t>(g, rows / beams, s);
    else launch_group<sps::bf16_t>(g, rows / beams, s);
    return sps::launch_status("sps_beam_select");
  }
  st = check_ws(workspace, workspace_bytes, parts_bytes(rows, sp, k), "sps_beam_select");
  if (st != SPS_OK) return st;
  sps::SelArgs a{};
  a.x = scores->data;
  a.ld = scores->ld;
  a.n_cols = scores->n_cols;
  a.col_begin = scores->col_begin;
  a.offsets = beam_scores;
  a.k = k;
  a.splits = sp.splits;
  a.seg = sp.seg;
  a.first = 1;
  a.parts = static_cast<uint64_t *>(workspace);
  launch_select(scores->dtype, a, rows, s);
  sps::JoinArgs j{};
  j.parts = a.parts;
  j.beams = beams;
  j.splits = sp.splits;
  j.k_in = k;
  j.k = k;
  j.scores = out_scores;
  j.parents = out_parents;
  j.cols = out_cols;
  hipLaunchKernelGGL(sps::beam_join_kernel, dim3((uint32_t)(rows / beams)), dim3(sps::kSelThreads),
                     0, s, j);
  return sps::launch_status("sps_beam_select");
}

sps_status sps_beam_join(const float *top_scores, const int32_t *top_cols, int64_t n_rows,
                         int32_t k_in, int32_t beams, int32_t k, float *out_scores,
                         int32_t *out_parents, int32_t *out_cols, void *stream) {
  if (n_rows < 0) return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "sps_beam_join: negative size");
  if (n_rows >= kMax31) return sps::set_error(SPS_ERR_OVERFLOW, "sizes must be below 2^31");
  sps_status st = check_k(k_in, "sps_beam_join");
  if (st == SPS_OK) st = check_k(k, "sps_beam_join");
  if (st == SPS_OK) st = check_beams(n_rows, beams, 1, k_in, "sps_beam_join");
  if (st != SPS_OK) return st;
  if (n_rows == 0) return SPS_OK;
  if (!top_scores || !top_cols || !out_scores || !out_parents || !out_cols)
    return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "sps_beam_join: NULL list or output");
  st = sps::check_grid(n_rows / beams, sps::kSelThreads, "sps_beam_join");
  if (st != SPS_OK) return st;
  sps::JoinArgs j{};
  j.in_scores = top_scores;
  j.in_cols = top_cols;
  j.beams = beams;
  j.splits = 1;
  j.k_in = k_in;
  j.k = k;
  j.scores = out_scores;
  j.parents = out_parents;
  j.cols = out_cols;
  hipLaunchKernelGGL(sps::beam_join_kernel, dim3((uint32_t)(n_rows / beams)),
                     dim3(sps::kSelThreads), 0, reinterpret_cast<hipStream_t>(stream), j);
  return sps::launch_status("sps_beam_join");
}

sps_status sps_reorder_states(const sps_state *states, int32_t n_states, const int32_t *parents,
                              int64_t n_out, int64_t n_rows, void *stream) {
  if (n_states < 0 || n_out < 0 || n_rows < 0)
    return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "sps_reorder_states: negative size");
  if (n_out >= kMax31 || n_rows >= kMax31)
    return sps::set_error(SPS_ERR_OVERFLOW, "sizes must be below 2^31");
  if (n_states == 0 || n_out == 0) return SPS_OK;
  if (!states || !parents)
    return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "sps_reorder_states: NULL argument");
  for (int32_t i = 0; i < n_states; ++i) {
    const sps_state &x = states[i];
    if (x.row_bytes < 0 || x.src_stride < x.row_bytes || x.dst_stride < x.row_bytes)
      return sps::set_error(SPS_ERR_INVALID_ARGUMENT,
                            "sps_reorder_states: state %d has a stride below its row", i);
    if (x.src_stride > INT64_MAX / 4 / (n_rows + 1) || x.dst_stride > INT64_MAX / 4 / (n_out + 1))
      return sps::set_error(SPS_ERR_OVERFLOW, "sps_reorder_states: state %d: rows x stride", i);
    if (x.row_bytes == 0) continue;
    if ((!x.src && n_rows > 0) || !x.dst)
      return sps::set_error(SPS_ERR_INVALID_ARGUMENT, "sps_reorder_states: state %d is NULL", i);
    if ((x.row_bytes + sps::kPieceBytes - 1) / sps::kPieceBytes > kMaxPieces / n_out)
      return sps::set_error(SPS_ERR_OVERFLOW, "sps_reorder_states: state %d exceeds a launch", i);
  }
  // sources are read while the destinations are written, and those in no order
  for (int32_t i = 0; i < n_states; ++i) {
    const sps_state &x = states[i];
    const sps::RowBytes dst{x.dst, n_out, x.row_bytes, x.dst_stride};
    if (sps::rows_overlap(dst, {parents, 1, n_out * 4, n_out * 4}))
      return sps::set_error(SPS_ERR_INVALID_ARGUMENT,
                            "sps_reorder_states: output %d overlaps the parents", i);
    for (int32_t j = 0; j < n_states; ++j) {
      const sps_state &y = states[j];
      if (sps::rows_overlap(dst, {y.src, n_rows, y.row_bytes, y.src_stride}))
        return sps::set_error(SPS_ERR_INVALID_ARGUMENT,
                              "sps_reorder_states: output %d overlaps state %d", i, j);
      if (j < i && sps::rows_overlap(dst, {y.dst, n_out, y.row_bytes, y.dst_stride}))
        return sps::set_error(SPS_ERR_INVALID_ARGUMENT,
                              "sps_reorder_states: output %d overlaps output %d", i, j);
    }
  }
  int32_t i = 0;
  while (i < n_states) {
    sps::StateArgs a{};
    a.parents = parents;
    a.n_rows = n_rows;
    int64_t blocks = 0;
    for (; i < n_states && a.n < sps::kMaxStates; ++i) {
      const sps_state &x = states[i];
      if (x.row_bytes == 0) continue;
      const int64_t pieces = (x.row_bytes + sps::kPieceBytes - 1) / sps::kPieceBytes;
      if (blocks + pieces * n_out > kMaxPieces) break;
      const int32_t k = a.n++;
      a.src[k] = static_cast<const uint8_t *>(x.src);
      a.dst[k] = static_cast<uint8_t *>(x.dst);
      a.bytes[k] = x.row_bytes;
      a.src_stride[k] = x.src_stride;
      a.dst_stride[k] = x.dst_stride;
      a.pieces[k] = (int32_t)pieces;
      a.first[k] = blocks;
      const uint64_t all = reinterpret_cast<uintptr_t>(x.src) | reinterpret_cast<uintptr_t>(x.dst) |
                           (uint64_t)x.row_bytes | (uint64_t)x.src_stride | (uint64_t)x.dst_stride;
      a.width[k] = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
      blocks += pieces * n_out;
    }
    a.first[a.n] = blocks;
    if (a.n > 0)
      hipLaunchKernelGGL(sps::reorder_kernel, dim3((uint32_t)blocks), dim3(256), 0,
                         reinterpret_cast<hipStream_t>(stream), a);
  }
  return sps::launch_status("sps_reorder_states");
}

}  // extern "C"
