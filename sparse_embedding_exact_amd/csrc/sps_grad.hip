// sps_grad.hip -- the gradient of the cosines with respect to the stored
// values of the sparse rows, on gfx950.
//
// Mathematics. With unit rows u (this side) and w (the other side) a score is
// S[r, i] = u_r . w_i, so entry e = (r, d) has du_e = sum_i G[r, i] w_i[d]:
// over the items that hold d, which is the posting list of d that scoring
// walks, with G gathered at the list's items in place of scores scattered to
// them. The norm's part follows once all chunks are in: dv = (du - u (u .
// du)) / |v|.
//
// Layout (of the walk over a prepared corpus). A workgroup keeps kGradRows
// rows of G over one slice (at most 1024
// items) in LDS and walks the lists of those rows' dims in that slice; every
// entry of a row gets one float32 sum a slice, in a fixed order, and a second
// pass adds the slices. G is read once; the lists come from the L2 of the XCD
// that works on the slice, since consecutive workgroups of an XCD take
// consecutive row groups of the same slice. 2000 queries x chunks of 8192 of
// the same corpus in turn: 134 us for the queries' side, 147 for the items',
// bound by the latency of short lists and by the loads of long ones, which
// every row walks for itself (rows of a workgroup do not share a list here, as
// they do in the walk of a whole matrix below).
#include "sps_rows.h"

namespace sps {

constexpr int kGradRows = 8;      // rows of a workgroup: 8 x 1028 floats are 33 KB of LDS
constexpr int kGradThreads = 256;
constexpr int kGradPitch = kSliceMax + 4;  // rows start 4 banks apart
constexpr int kGradShort = 4;     // a list of at most this many postings is one lane's

struct WalkArgs {
  const int32_t *indptr, *indices;
  int64_t nnz, n_rows, n_groups;
  Geom g;
  int32_t chunk;
  const int4 *dinfo;
  const uint4 *dtab;
  const uint2 *post;
  const int32_t *slice_base;
  const void *grad;
  int64_t ld;
  int32_t transposed, first;
  float *du;     // one slice a chunk: the sums go here
  float *parts;  // else [slice][entry]
};

// Workgroup b of T in the order of the tiles: XCD b % 8 takes one contiguous
// run of them (hardware hands workgroups to the XCDs in turn).
__device__ __forceinline__ int64_t xcd_tile(int64_t b, int64_t total) {
  const int64_t q = total / 8, r = total % 8, x = b % 8;
  return x * q + (x < r ? x : r) + b / 8;
}

// Sum of a float over the row of 16 lanes (in its last lane), and over the
// wave (in lane 63); every lane must be active.
template <int CTRL, int ROW_MASK, bool BOUND>
__device__ __forceinline__ float dpp_f32(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL,
                                                               ROW_MASK, 0xf, BOUND));
}
__device__ __forceinline__ float row16_total(float x) {
  x += dpp_f32<0x111, 0xf, true>(x);   // row_shr:1
  x += dpp_f32<0x112, 0xf, true>(x);   // row_shr:2
  x += dpp_f32<0x114, 0xf, true>(x);   // row_shr:4
  x += dpp_f32<0x118, 0xf, true>(x);   // row_shr:8
  return x;
}
__device__ __forceinline__ float wave_total(float x) {
  x = row16_total(x);
  x += dpp_f32<0x142, 0xa, false>(x);  // row_bcast:15
  x += dpp_f32<0x143, 0xc, false>(x);  // row_bcast:31
  return x;
}

template <typename T>
__global__ __launch_bounds__(kGradThreads) void grad_walk_kernel(WalkArgs a) {
  __shared__ float tile[kGradRows][kGradPitch];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t id = xcd_tile(blockIdx.x, gridDim.x);
  const int32_t sub = (int32_t)(id / a.n_groups);
  const int64_t r0 = (id % a.n_groups) * kGradRows;
  const int nr = a.n_rows - r0 < kGradRows ? (int)(a.n_rows - r0) : kGradRows;
  const int64_t sl = (int64_t)a.chunk * a.g.n_sub + sub;
  const int64_t sb = a.g.slice_begin(sl) - a.g.chunk_begin(a.chunk);
  const int len = (int)(a.g.slice_end(sl) - a.g.slice_begin(sl));
  const T *grad = static_cast<const T *>(a.grad);
  constexpr int V = kVec<T>;
  if (!a.transposed) {
    for (int r = wave; r < nr; r += kGradThreads / 64) {
      const T *p = grad + (r0 + r) * a.ld + sb;
      for (int j = lane * V; j < len; j += 64 * V) {
        if (j + V <= len) {
          const Vec<T> v = *reinterpret_cast<const Vec<T> *>(p + j);
#pragma unroll
          for (int e = 0; e < V; ++e) tile[r][j + e] = to_f32(v.e[e]);
        } else {
          for (int e = 0; j + e < len; ++e) tile[r][j + e] = to_f32(p[j + e]);
        }
      }
    }
  } else {
    const int r = t % kGradRows;
    if (r < nr)
      for (int j = t / kGradRows; j < len; j += kGradThreads / kGradRows)
        tile[r][j] = to_f32(grad[(sb + j) * a.ld + r0 + r]);
  }
  __syncthreads();
  const int4 info = a.dinfo[sl];
  const int32_t base = a.slice_base[sl];
  const int32_t snnz = a.slice_base[sl + 1] - base;
  const uint2 *post = a.post + base;
  for (int r = wave; r < nr; r += kGradThreads / 64) {
    const int64_t e0 = clamp64(a.indptr[r0 + r], 0, a.nnz);
    const int64_t e1 = clamp64(a.indptr[r0 + r + 1], e0, a.nnz);
    const float *g = tile[r];
    for (int64_t w0 = e0; w0 < e1; w0 += 64) {
      const int64_t e = w0 + lane;
      int32_t start = 0, n = 0;
      if (e < e1) {
        if (!dim_lookup(a.dtab, info, (uint32_t)a.indices[e], start, n)) n = 0;
        if (start < 0 || n > snnz - start) n = 0;
      }
      float acc = 0;
      if (n > 0 && n <= kGradShort) {
        uint2 p[kGradShort];
#pragma unroll
        for (int i = 0; i < kGradShort; ++i) p[i] = post[start + (i < n ? i : 0)];
#pragma unroll
        for (int i = 0; i < kGradShort; ++i) {
          const float x = g[p[i].x & (kSliceMax - 1)];
          acc += i < n ? x * __builtin_bit_cast(float, p[i].y) : 0.0f;
        }
      }
      uint64_t rest = __ballot(n > kGradShort);
      while (rest) {
        const int l = __builtin_ctzll(rest);
        rest &= rest - 1;
        const int32_t s = __builtin_amdgcn_readlane(start, l);
        const int32_t m = __builtin_amdgcn_readlane(n, l);
        float part = 0;
        for (int i = lane; i < m; i += 256) {
          uint2 p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = post[s + (i + 64 * j < m ? i + 64 * j : i)];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = g[p[j].x & (kSliceMax - 1)];
            part += i + 64 * j < m ? x * __builtin_bit_cast(float, p[j].y) : 0.0f;
          }
        }
        part = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wave_total(part)), 63));
        if (lane == l) acc = part;
      }
      if (e < e1) {
        if (a.parts) a.parts[sub * a.nnz + e] = acc;
        else a.du[e] = a.first ? acc : a.du[e] + acc;
      }
    }
  }
}

// du[e] += the slices' sums, in the order of the slices.
__global__ __launch_bounds__(256) void grad_fold_kernel(WalkArgs a) {
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < a.nnz;
       e += (int64_t)gridDim.x * 256) {
    float s = a.first ? 0.0f : a.du[e];
    for (int j = 0; j < a.g.n_sub; ++j) s += a.parts[j * a.nnz + e];
    a.du[e] = s;
  }
}

// dv of the entries [e0, e1) of a row from its du, by one wave; sums in float64.
__device__ __forceinline__ void through_norm(const float *__restrict__ values, const float *du,
                                             float *dv, int64_t e0, int64_t e1, int lane) {
  double nn = 0, dot = 0;
  for (int64_t e = e0 + lane; e < e1; e += 64) {
    const double v = values[e];
    nn += v * v;
    dot += v * (double)du[e];
  }
  nn = wave_sum(nn);
  dot = wave_sum(dot);
  const double inv = nn > 0 ? 1.0 / sqrt(nn) : 0.0, along = nn > 0 ? dot / nn : 0.0;
  for (int64_t e = e0 + lane; e < e1; e += 64)
    dv[e] = nn > 0 ? (float)(((double)du[e] - (double)values[e] * along) * inv) : 0.0f;
}

// One wave a row.
__global__ __launch_bounds__(256) void grad_values_kernel(int64_t n_rows, int64_t nnz,
                                                          const int32_t *__restrict__ indptr,
                                                          const float *__restrict__ values,
                                                          const float *du, float *dv) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= n_rows) return;  // uniform per wave
  const int64_t e0 = clamp64(indptr[row], 0, nnz), e1 = clamp64(indptr[row + 1], e0, nnz);
  through_norm(values, du, dv, e0, e1, threadIdx.x & 63);
}

// ---------------------------------------------------------------------------
// Both sides of a whole score matrix, from the two CSRs alone.
//
// The lists that a side walks are the other side's entries by dim. They are
// made here by a stable radix sort of both CSRs at once (dim as the key, row
// and unit value as the load), not taken from a prepared corpus: a training
// step has new values every time, its batches are small, and a corpus'
// per-slice sorts and dim index would keep 8 to 16 workgroups busy for longer
// than all that follows. Unit values with the first histogram; a prefix and a
// scatter a pass of up to 11 bits, a histogram for each pass but the first; the
// table of the lists; the walk: 2 + 3 launches a pass, 5 for dims up to 2^11, 8
// up to 2^22, 11 beyond.
//
// Rows are canonical: dims ascend and differ. A row whose dims do not gives
// undefined gradients (the bisection for a dim's mates misses some), but places
// and columns are clamped or masked, so that nothing out of range is accessed.
//
// The walk keeps four rows of G over 4096 columns in LDS, the four values of a
// column side by side, and gives each entry of its rows a lane, which looks the
// entry's list up. Lists of up to 4 entries are the lane's own,
// of up to 128 a group of 16 lanes'. A longer one is a wave's, 512 entries in
// flight, and serves every row of the four that holds the dim: such dims are
// the ones that most rows share, one load of an entry and one 16-byte read of
// LDS then make four products. The norm's part is taken off at the end of the
// same launch.
//
// Measured: 2000 x 8192, 43 entries a row, Zipf(1.1): 193 us, of which unit
// values and sort 45, table 9, walk 142 (without the long lists 80, without
// the group lists 128, without loading G, which the items' side reads 16 bytes
// of a row at a time, 117, with none of these 18). Long lists are bound by the
// loads of their entries and the gathers from LDS: vector issue is busy for
// half of the walk and LDS for 37 %, half of it bank conflicts, and 93 % of
// the loads hit in L2 (1001 x 8192). More of them in flight (1024, or a next
// 512 loaded ahead), four lists a wave at a time and lists handed to whichever
// wave is free were no faster, half the bank conflicts (8-byte loads of
// neighbouring entries) 10 % slower. Rows one at a time, without the sharing,
// took 335 us, prepared corpora instead of the sort 1488.
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxBits = 11;
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kSortMinEntries = 2048;  // of a workgroup, at least
constexpr int kSortBlocks = 250;       // about: one a CU
constexpr int kSortAhead = 16;         // entries of a lane in flight
constexpr int kPrefixWaves = 16, kPrefixEach = 16;
static_assert(kPrefixWaves * kPrefixEach > kSortBlocks, "a side has at most kSortBlocks + 1 blocks");
constexpr int kWalkThreads = 512;
constexpr int kWalkWaves = kWalkThreads / 64;
constexpr int kWalkRows = 4;           // rows of G side by side in LDS
constexpr int kWalkCols = 4096;        // and their columns: 64 KB, two workgroups a CU
constexpr int kBatch = kWalkThreads;   // entries walked at a time, one a thread
constexpr int kFillEach = 8;           // slots of a thread that empties them
constexpr int kLaneList = 4, kGroupList = 128;

struct BothSide {
  const int32_t *indptr, *indices;
  const float *values;
  float *dv;
  int64_t n_rows, nnz;
  int64_t base;       // of its entries in the joint arrays
  int32_t block0, blocks;  // of the sort
  uint4 *lists;            // slots of its dims: (dim, first place, place behind the last, -)
  uint32_t slots;
  int64_t groups;
};

struct BothArgs {
  BothSide s[2];  // queries, items
  float *unit;    // [entries of both]: value / norm
  int32_t *row;   // row of the entry
  int32_t *key[2];
  uint2 *load[2]; // (row, bits of the unit value)
  int32_t *hist;  // [sort blocks][bins]
  int32_t *total; // [sides][kMaxBins]
  int64_t per_block;
  int32_t pass, passes, bits, last;  // `last`: which of the buffers holds the lists
  const void *grad;
  int64_t ld;
};

__device__ __forceinline__ int digit_of(int32_t key, const BothArgs &a) {
  return (int)((uint32_t)key >> (a.pass * a.bits)) & ((1 << a.bits) - 1);
}

// the entries of sort block b: side, and joint positions [lo, hi)
__device__ __forceinline__ int sort_range(const BothArgs &a, int b, int64_t &lo, int64_t &hi) {
  const int side = b >= a.s[1].block0;
  const BothSide &s = a.s[side];
  lo = s.base + (int64_t)(b - s.block0) * a.per_block;
  hi = lo + a.per_block < s.base + s.nnz ? lo + a.per_block : s.base + s.nnz;
  return side;
}
__device__ __forceinline__ int32_t key_at(const BothArgs &a, int side, int64_t e) {
  return a.pass == 0 ? a.s[side].indices[e - a.s[side].base] : a.key[(a.pass - 1) & 1][e];
}

__device__ __forceinline__ void histogram(const BothArgs &a, int b, int32_t *cnt) {
  const int bins = 1 << a.bits;
  for (int i = threadIdx.x; i < bins; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  int64_t lo, hi;
  const int side = sort_range(a, b, lo, hi);
  for (int64_t e0 = lo + threadIdx.x; e0 < hi; e0 += kSortThreads * kSortAhead) {
    int32_t k[kSortAhead];
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i) {
      const int64_t e = e0 + (int64_t)i * kSortThreads;
      k[i] = key_at(a, side, e < hi ? e : e0);
    }
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i)
      if (e0 + (int64_t)i * kSortThreads < hi) atomicAdd(&cnt[digit_of(k[i], a)], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < bins; i += kSortThreads) a.hist[(int64_t)b * bins + i] = cnt[i];
}

// Unit values and row numbers, one wave a row; the first workgroups make the
// first histogram and the last ones empty the slots, which need neither.
__global__ __launch_bounds__(kSortThreads) void both_unit_kernel(BothArgs a) {
  __shared__ int32_t cnt[kMaxBins];
  const int blocks = a.s[0].blocks + a.s[1].blocks;
  if ((int)blockIdx.x < blocks) {
    histogram(a, blockIdx.x, cnt);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t row_blocks = (a.s[0].n_rows + a.s[1].n_rows + kSortWaves - 1) / kSortWaves;
  int64_t row = (int64_t)(blockIdx.x - blocks) * kSortWaves + (threadIdx.x >> 6);
  if ((int64_t)blockIdx.x - blocks >= row_blocks) {  // both sides' slots are one array
    const int64_t first = (int64_t)blockIdx.x - blocks - row_blocks;
    const int64_t n = (int64_t)a.s[0].slots + a.s[1].slots;
    for (int i = 0; i < kFillEach; ++i) {
      const int64_t j = (first * kFillEach + i) * kSortThreads + threadIdx.x;
      if (j < n) a.s[0].lists[j] = make_uint4(kDimEmpty, 0, 0, 0);
    }
    return;
  }
  int side = 0;
  if (row >= a.s[0].n_rows) {
    row -= a.s[0].n_rows;
    side = 1;
  }
  const BothSide &s = a.s[side];
  if (row >= s.n_rows) return;
  const int64_t e0 = clamp64(s.indptr[row], 0, s.nnz), e1 = clamp64(s.indptr[row + 1], e0, s.nnz);
  double nn = 0;
  for (int64_t e = e0 + lane; e < e1; e += 64) nn += (double)s.values[e] * (double)s.values[e];
  nn = wave_sum(nn);
  const double inv = nn > 0 ? 1.0 / sqrt(nn) : 0.0;
  for (int64_t e = e0 + lane; e < e1; e += 64) {
    a.unit[s.base + e] = (float)((double)s.values[e] * inv);
    a.row[s.base + e] = (int32_t)row;
  }
}

__global__ __launch_bounds__(kSortThreads) void both_hist_kernel(BothArgs a) {
  __shared__ int32_t cnt[kMaxBins];
  histogram(a, blockIdx.x, cnt);
}

// Per side and digit: the blocks' counts become the counts of the blocks
// before them, and their sum goes to `total`. A workgroup takes 64 digits, a
// sixteenth of the blocks each wave, whose counts are all on their way at once:
// the launch is bound by that one round trip (4 waves that read twice, eight at
// a time: 7.7 us instead of 4.7 at 2000 x 8192). Every scatter block adding
// up all histograms by itself took 14 of its 26 us at 440,000 entries: the
// counts have just been written by other XCDs.
__global__ __launch_bounds__(kPrefixWaves * 64) void both_prefix_kernel(BothArgs a) {
  __shared__ int32_t part[kPrefixWaves][64];
  const int bins = 1 << a.bits, lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int per_side = (bins + 63) / 64;
  const int side = (int)blockIdx.x / per_side;
  const int d = (int)blockIdx.x % per_side * 64 + lane;
  const BothSide &s = a.s[side];
  const int j0 = q * kPrefixEach;
  int32_t *h = a.hist + (int64_t)s.block0 * bins + (d < bins ? d : 0);
  int32_t c[kPrefixEach], sum = 0;
#pragma unroll
  for (int j = 0; j < kPrefixEach; ++j) c[j] = j0 + j < s.blocks ? h[(int64_t)(j0 + j) * bins] : 0;
#pragma unroll
  for (int j = 0; j < kPrefixEach; ++j) sum += c[j];
  part[q][lane] = sum;
  __syncthreads();
  int32_t at = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kPrefixWaves; ++i) {
    const int32_t v = part[i][lane];
    at += i < q ? v : 0;
    total += v;
  }
  if (d >= bins) return;
#pragma unroll
  for (int j = 0; j < kPrefixEach; ++j) {
    if (j0 + j < s.blocks) h[(int64_t)(j0 + j) * bins] = at;
    at += c[j];
  }
  if (q == 0) a.total[side * kMaxBins + d] = total;
}

// Stable: a block's entries are cut among its waves in order, a wave takes 64
// at a time, and equal digits among them are ranked by lane. Entries counted
// last are placed first, from registers: 10.6 us a pass at 2000 x 8192, loaded
// again 11.8. What bounds it then is the two stores of an entry, to a line each.
__global__ __launch_bounds__(kSortThreads) void both_scatter_kernel(BothArgs a) {
  __shared__ int32_t cnt[kSortWaves][kMaxBins];
  __shared__ int32_t ws[kSortWaves];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, b = blockIdx.x;
  const int bins = 1 << a.bits;
  int64_t lo, hi;
  const int side = sort_range(a, b, lo, hi);
  const BothSide &s = a.s[side];
  const int64_t part = ((a.per_block / kSortWaves) + 63) / 64 * 64;
  const int64_t e0 = lo + w * part < hi ? lo + w * part : hi;
  const int64_t e1 = w + 1 < kSortWaves && e0 + part < hi ? e0 + part : hi;
  const uint2 *from = a.load[(a.pass + 1) & 1];
  int32_t k[kSortAhead];
  uint2 v[kSortAhead];
  const auto keys = [&](int64_t w0) {
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i) {
      const int64_t x = w0 + 64 * i + lane;
      k[i] = key_at(a, side, x < e1 ? x : w0);
    }
  };
  const auto loads = [&](int64_t w0) {
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i) {
      const int64_t x = w0 + 64 * i + lane, e = x < e1 ? x : w0;
      v[i] = a.pass == 0 ? make_uint2((uint32_t)a.row[e], __builtin_bit_cast(uint32_t, a.unit[e]))
                         : from[e];
    }
  };
  // counted from the last 1024 entries of the wave to the first, which stay in registers
  const int64_t turns = e1 > e0 ? (e1 - e0 - 1) / (64 * kSortAhead) : 0;
  // thread t places digits 4 t .. 4 t + 3
  int32_t total[4] = {}, before[4] = {};
  if (4 * t < bins) {
    const int4 v = *reinterpret_cast<const int4 *>(a.total + side * kMaxBins + 4 * t);
    const int4 h = *reinterpret_cast<const int4 *>(a.hist + (int64_t)b * bins + 4 * t);
    total[0] = v.x, total[1] = v.y, total[2] = v.z, total[3] = v.w;
    before[0] = h.x, before[1] = h.y, before[2] = h.z, before[3] = h.w;
  }
  for (int i = lane; i < bins; i += 64) cnt[w][i] = 0;
  for (int64_t n = turns; n >= 0 && e0 < e1; --n) {
    const int64_t w0 = e0 + n * 64 * kSortAhead;
    keys(w0);
    if (n == 0) loads(w0);
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i)
      if (w0 + 64 * i + lane < e1) atomicAdd(&cnt[w][digit_of(k[i], a)], 1);
  }
  __syncthreads();
  int32_t all;
  const int32_t sum = total[0] + total[1] + total[2] + total[3];
  int32_t at = block_incl_scan<kSortThreads, int32_t>(sum, ws, &all) - sum + (int32_t)s.base;
  if (4 * t < bins)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int32_t o = at + before[i];
#pragma unroll
      for (int j = 0; j < kSortWaves; ++j) {
        const int32_t c = cnt[j][4 * t + i];
        cnt[j][4 * t + i] = o;
        o += c;
      }
      at += total[i];
    }
  __syncthreads();
  int32_t *key = a.key[a.pass & 1];
  uint2 *load = a.load[a.pass & 1];
  for (int64_t w0 = e0; w0 < e1; w0 += 64 * kSortAhead) {
    if (w0 > e0) {
      keys(w0);
      loads(w0);
    }
#pragma unroll
    for (int i = 0; i < kSortAhead; ++i) {
      if (w0 + 64 * i >= e1) break;  // uniform
      const bool valid = w0 + 64 * i + lane < e1;
      const int d = digit_of(k[i], a);
      uint64_t same = __ballot(valid);
      for (int j = 0; j < a.bits; ++j) {
        const bool bit = d >> j & 1;
        const uint64_t m = __ballot(bit);
        same &= bit ? m : ~m;
      }
      if (valid) {
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int32_t p = cnt[w][d] + rank;
        __builtin_amdgcn_wave_barrier();
        if (rank == 0) cnt[w][d] = p + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        key[p] = k[i];
        load[p] = v[i];
      }
    }
  }
}

// Where a dim's entries stand among a side's sorted ones: an open-addressing
// table, filled by the threads of each run's first and last entry (whichever
// comes first takes the slot). Slots outnumber the entries, so that a chain
// ends; where a dim lies in the table depends on the order of insertion and is
// never observed. A lookup is one or two loads, where a bisection of the keys
// is eighteen dependent ones.
__device__ __forceinline__ uint32_t slot_of(uint32_t d, uint32_t slots) {
  return (uint32_t)(((uint64_t)(d * 0x9E3779B1u) * slots) >> 32);
}
__global__ __launch_bounds__(256) void both_lists_kernel(BothArgs a) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int side = p >= a.s[1].base;
  const BothSide &s = a.s[side];
  const int64_t e = s.base + s.nnz;
  if (p >= e) return;
  const int32_t *key = a.key[a.last];
  const uint32_t d = (uint32_t)key[p];
  const bool first = p == s.base || (uint32_t)key[p - 1] != d;
  const bool last = p + 1 == e || (uint32_t)key[p + 1] != d;
  if (!first && !last) return;
  uint32_t *slot = reinterpret_cast<uint32_t *>(s.lists);
  uint32_t i = slot_of(d, s.slots);
  for (uint32_t n = 0; n < s.slots; ++n) {
    const uint32_t was = atomicCAS(slot + 4 * (int64_t)i, kDimEmpty, d);
    if (was == kDimEmpty || was == d) {
      if (first) slot[4 * (int64_t)i + 1] = (uint32_t)p;
      if (last) slot[4 * (int64_t)i + 2] = (uint32_t)(p + 1);
      return;
    }
    i = i + 1 == s.slots ? 0 : i + 1;
  }
}
__device__ __forceinline__ void find_list(const BothSide &s, uint32_t d, int32_t &l, int32_t &h) {
  uint32_t i = slot_of(d, s.slots);
  for (uint32_t n = 0; n < s.slots; ++n) {
    const uint4 v = s.lists[i];
    if (v.x == d) {
      l = (int32_t)v.y;
      h = (int32_t)v.z;
      return;
    }
    if (v.x == kDimEmpty) return;
    i = i + 1 == s.slots ? 0 : i + 1;
  }
}

struct BothShared {
  float4 tile[kWalkCols];  // indexes are masked: in range whatever a CSR holds
  int32_t dim[kBatch];
  float acc[kBatch], value[kBatch];
  int32_t begin[kWalkRows + 1];  // of the rows' entries in the batch
};
static_assert(kWalkRows == 4, "the rows of G are a float4");

// two entries, 8-byte aligned
struct __attribute__((packed, aligned(8))) Pair {
  uint2 a, b;
};

// Up to 128 N entries of a list from q on (this lane: q, q + 1, and every 128
// further), times the four rows' values of their columns; none at or past h.
// Lanes past h take the last entry times zero: where G is infinite there, NaN
// stands in place of an infinity, in rows that the norm's part leaves without a
// finite gradient either way.
template <int N, bool WHOLE>
__device__ __forceinline__ void four_rows(const uint2 *load, int32_t q, int32_t h, uint32_t c0,
                                          const float4 *tile, float4 &s) {
  Pair v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (WHOLE) {
      v[k] = *reinterpret_cast<const Pair *>(load + q + k * 128);
    } else {
      const int32_t j = q + k * 128;
      v[k].a = load[j < h ? j : h - 1];
      v[k].b = load[j + 1 < h ? j + 1 : h - 1];
      if (j >= h) v[k].a.y = 0;
      if (j + 1 >= h) v[k].b.y = 0;
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float4 ga = tile[(v[k].a.x - c0) & (kWalkCols - 1)];
    const float4 gb = tile[(v[k].b.x - c0) & (kWalkCols - 1)];
    const float wa = __builtin_bit_cast(float, v[k].a.y), wb = __builtin_bit_cast(float, v[k].b.y);
    s.x += ga.x * wa;
    s.y += ga.y * wa;
    s.z += ga.z * wa;
    s.w += ga.w * wa;
    s.x += gb.x * wb;
    s.y += gb.y * wb;
    s.z += gb.z * wb;
    s.w += gb.w * wb;
  }
}

template <typename T, bool TRANSPOSED>
__device__ __forceinline__ void walk(const BothArgs &a, int side, int64_t group, BothShared &sh) {
  const BothSide &s = a.s[side], &o = a.s[1 - side];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int64_t r0 = group * kWalkRows;
  const int nr = s.n_rows - r0 < kWalkRows ? (int)(s.n_rows - r0) : kWalkRows;
  const int64_t e0 = clamp64(s.indptr[r0], 0, s.nnz), e1 = clamp64(s.indptr[r0 + nr], e0, s.nnz);
  const uint2 *load = a.load[a.last];
  const T *g = static_cast<const T *>(a.grad);
  const float *tile1 = reinterpret_cast<const float *>(sh.tile);
  for (int64_t eb = e0; eb < e1; eb += kBatch) {
    const int ne = e1 - eb < kBatch ? (int)(e1 - eb) : kBatch;
    __syncthreads();  // the batch before is done with
    if (t <= nr) {
      const int64_t b = clamp64(s.indptr[r0 + t], e0, e1) - eb;
      sh.begin[t] = (int32_t)clamp64(b, 0, ne);
    }
    // entry i is thread (i % 8) * 64 + i / 8's: every wave gets some of a short row
    const int i = lane * kWalkWaves + w;
    int32_t l = 0, h = 0, row = 0;
    if (i < ne) {
      const int32_t d = s.indices[eb + i];
      sh.value[i] = s.values[eb + i];
      find_list(o, (uint32_t)d, l, h);
      sh.dim[i] = d;
      sh.acc[i] = 0;
    }
    __syncthreads();
    if (i < ne)
      for (int r = 1; r < nr; ++r) row += i >= sh.begin[r];
    // a long list: the first row that has the dim walks it, for the others too
    uint32_t mate01 = ~0u, mate23 = ~0u;  // each row's entry, 16 bits each, all ones for none
    bool leads = false;
    if (i < ne && h - l > kGroupList) {
      const int32_t d = sh.dim[i];
      int32_t x0[kWalkRows], x1[kWalkRows];  // bisections of the rows' ascending dims
#pragma unroll
      for (int r = 0; r < kWalkRows; ++r) {
        x0[r] = r < nr ? sh.begin[r] : 0;
        x1[r] = r < nr ? sh.begin[r + 1] : 0;
      }
      bool more = true;
      while (more) {
        more = false;
#pragma unroll
        for (int r = 0; r < kWalkRows; ++r)
          if (x0[r] < x1[r]) {
            const int32_t x = (x0[r] + x1[r]) >> 1;
            if (sh.dim[x] < d) x0[r] = x + 1;
            else x1[r] = x;
            more = true;
          }
      }
      leads = true;
      uint32_t m[kWalkRows];
#pragma unroll
      for (int r = 0; r < kWalkRows; ++r) {
        const bool has = r < nr && x0[r] < sh.begin[r + 1] && sh.dim[x0[r]] == d;
        m[r] = has ? (uint32_t)x0[r] : 0xFFFFu;
        if (has && r < row) leads = false;
      }
      mate01 = m[0] | m[1] << 16;
      mate23 = m[2] | m[3] << 16;
      if (!leads) h = l;
    }
    for (int64_t c0 = 0; c0 < o.n_rows; c0 += kWalkCols) {
      const int nc = o.n_rows - c0 < kWalkCols ? (int)(o.n_rows - c0) : kWalkCols;
      __syncthreads();
#pragma unroll 4
      for (int c = t; c < nc; c += kWalkThreads) {
        float v[kWalkRows];
        if (!TRANSPOSED) {
          const T *p = g + r0 * a.ld + c0 + c;
#pragma unroll
          for (int r = 0; r < kWalkRows; ++r) v[r] = r < nr ? to_f32(p[r * a.ld]) : 0.0f;
        } else {
          const T *p = g + (c0 + c) * a.ld + r0;
          if (nr == kWalkRows) {
            struct __attribute__((packed, aligned(sizeof(T)))) Four {
              T e[kWalkRows];
            };
            const Four q = *reinterpret_cast<const Four *>(p);
#pragma unroll
            for (int r = 0; r < kWalkRows; ++r) v[r] = to_f32(q.e[r]);
          } else {
#pragma unroll
            for (int r = 0; r < kWalkRows; ++r) v[r] = r < nr ? to_f32(p[r]) : 0.0f;
          }
        }
        sh.tile[c] = make_float4(v[0], v[1], v[2], v[3]);
      }
      __syncthreads();
      // the list's part in this tile starts where the last tile's ended. A lane's own few entries
      // are looked at in every tile instead, each for its column; a leading list is cut to the
      // last entry, since the wave that walks it asks for no column
      const bool cut = nc < o.n_rows && (leads ? h > l : h - l > kLaneList);
      int32_t next = h;
      if (cut) {
        int32_t m0 = l, m1 = h;
        while (m0 < m1) {
          const int32_t m = m0 + ((m1 - m0) >> 1);
          if ((int64_t)load[m].x < c0 + nc) m0 = m + 1;
          else m1 = m;
        }
        next = m0;
      }
      const int n = next - l;
      float acc = 0;
      if (!leads && n > 0 && n <= kLaneList) {
        uint2 v[kLaneList];
#pragma unroll
        for (int j = 0; j < kLaneList; ++j) v[j] = load[l + (j < n ? j : 0)];
#pragma unroll
        for (int j = 0; j < kLaneList; ++j) {
          const uint32_t c = v[j].x - (uint32_t)c0;  // may lie in another tile
          const float x = tile1[(c & (kWalkCols - 1)) * kWalkRows + row];
          acc += j < n && c < (uint32_t)nc ? x * __builtin_bit_cast(float, v[j].y) : 0.0f;
        }
        sh.acc[i] += acc;
      }
      // four lists at a time, 16 lanes each
      uint64_t mid = __ballot(!leads && n > kLaneList);
      while (mid) {
        int src = -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int f = mid ? __builtin_ctzll(mid) : -1;
          if (k == lane >> 4) src = f;
          mid &= mid ? mid - 1 : 0;
        }
        const int from = src < 0 ? 0 : src;
        // every lane shuffles: a source lane must be active
        const int32_t l2 = __shfl(l, from, 64), n1 = __shfl(n, from, 64);
        const int row2 = __shfl(row, from, 64);
        const int32_t n2 = src < 0 ? 0 : n1;
        float part = 0;
        for (int q = lane & 15; q < n2; q += 64) {
          uint2 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = load[l2 + (q + 16 * k < n2 ? q + 16 * k : q)];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x =
                tile1[((v[k].x - (uint32_t)c0) & (kWalkCols - 1)) * kWalkRows + row2];
            part += q + 16 * k < n2 ? x * __builtin_bit_cast(float, v[k].y) : 0.0f;
          }
        }
        part = row16_total(part);
        if ((lane & 15) == 15 && src >= 0) sh.acc[src * kWalkWaves + w] += part;
      }
      // the whole wave's, for up to four rows
      uint64_t big = __ballot(leads && n > 0);
      while (big) {
        const int f = __builtin_ctzll(big);
        big &= big - 1;
        const int32_t l2 = __builtin_amdgcn_readlane(l, f), h2 = __builtin_amdgcn_readlane(next, f);
        const uint32_t m01 = (uint32_t)__builtin_amdgcn_readlane((int)mate01, f);
        const uint32_t m23 = (uint32_t)__builtin_amdgcn_readlane((int)mate23, f);
        float4 p = make_float4(0, 0, 0, 0);
        int32_t q = l2;
        for (; q + 512 <= h2; q += 512)
          four_rows<4, true>(load, q + lane * 2, h2, (uint32_t)c0, sh.tile, p);
        if (h2 - q > 256) four_rows<4, false>(load, q + lane * 2, h2, (uint32_t)c0, sh.tile, p);
        else if (h2 - q > 128) four_rows<2, false>(load, q + lane * 2, h2, (uint32_t)c0, sh.tile, p);
        else if (h2 > q) four_rows<1, false>(load, q + lane * 2, h2, (uint32_t)c0, sh.tile, p);
        p.x = wave_total(p.x);
        p.y = wave_total(p.y);
        p.z = wave_total(p.z);
        p.w = wave_total(p.w);
        if (lane == 63) {
          const uint32_t m[kWalkRows] = {m01 & 0xFFFFu, m01 >> 16, m23 & 0xFFFFu, m23 >> 16};
          const float x[kWalkRows] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int r = 0; r < kWalkRows; ++r)
            if (m[r] != 0xFFFFu) sh.acc[m[r]] += x[r];
        }
      }
      if (cut) l = next;
    }
    __syncthreads();
    if (e1 - e0 <= kBatch) {  // the rows are whole: the norm's part from LDS
      for (int r = w; r < nr; r += kWalkWaves)
        through_norm(sh.value, sh.acc, s.dv + eb, sh.begin[r], sh.begin[r + 1], lane);
      return;
    }
    if (i < ne) s.dv[eb + i] = sh.acc[i];
  }
  __syncthreads();
  for (int r = w; r < nr; r += kWalkWaves) {
    const int64_t b0 = clamp64(s.indptr[r0 + r], 0, s.nnz), b1 = clamp64(s.indptr[r0 + r + 1], b0, s.nnz);
    through_norm(s.values, s.dv, s.dv, b0, b1, lane);
  }
}

// Each XCD takes a run of the queries' groups, then one of the items'.
template <typename T>
__global__ __launch_bounds__(kWalkThreads) void both_walk_kernel(BothArgs a) {
  __shared__ BothShared sh;
  const int64_t b = blockIdx.x, first = (a.s[0].groups + 7) / 8 * 8;
  if (b < a.s[0].groups) walk<T, false>(a, 0, xcd_tile(b, a.s[0].groups), sh);
  else if (b >= first) walk<T, true>(a, 1, xcd_tile(b - first, a.s[1].groups), sh);
}

}  // namespace sps

namespace {

using sps::set_error;
constexpr int64_t kMax31 = 2147483647ll;

sps_status check_csr(const sps_csr *m, const char *what) {
  if (!m) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL CSR", what);
  if (m->n_rows < 0 || m->n_cols <= 0 || m->nnz < 0)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: negative size or n_cols <= 0", what);
  if (m->n_rows >= kMax31 || m->n_cols >= kMax31 || m->nnz >= kMax31)
    return set_error(SPS_ERR_OVERFLOW, "%s: sizes must be below 2^31", what);
  if (!m->indptr) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL indptr", what);
  if (m->nnz > 0 && (!m->indices || !m->values))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL indices or values", what);
  return SPS_OK;
}

// Slots of a side's table: more than its entries; for small sides many more,
// where the longest chain of a wave, not the table's size, is what costs (1.5
// slots an entry at 82,000 entries of 47,000 dims: 20 us to fill, 8: 6 us).
constexpr size_t kMoreSlots = 1 << 19;
uint32_t slots_of(int64_t nnz) {
  const int64_t least = nnz + nnz / 2, most = 8 * nnz;
  const int64_t more = most < (int64_t)kMoreSlots ? most : (int64_t)kMoreSlots;
  return (uint32_t)((least > more ? least : more) + 64);
}

struct BothLayout {
  size_t unit, row, key[2], load[2], sums, lists, hist, total;
  int64_t per_block;
};
BothLayout both_layout(int64_t n) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  BothLayout L;
  size_t at = 0;
  L.unit = at;
  at = up(at + (size_t)n * 4);
  L.row = at;
  at = up(at + (size_t)n * 4);
  for (int i = 0; i < 2; ++i) {
    L.key[i] = at;
    at = up(at + (size_t)n * 4);
    L.load[i] = at;
    at = up(at + (size_t)n * 8);
  }
  L.per_block = (n + sps::kSortBlocks - 1) / sps::kSortBlocks;
  if (L.per_block < sps::kSortMinEntries) L.per_block = sps::kSortMinEntries;
  L.lists = at;
  at = up(at + ((size_t)n + (size_t)n / 2 + 2 * kMoreSlots + 128) * 16);
  L.sums = at;
  at = up(at + 2 * sps::kMaxBins * 4);
  L.hist = at;
  // one block more on each side than full blocks of the whole
  at = up(at + ((size_t)(n / L.per_block) + 2) * sps::kMaxBins * 4);
  L.total = at;
  return L;
}

}  // namespace

extern "C" {

sps_status sps_cosine_grad_workspace_size(int64_t nnz, const sps_items *other, size_t *bytes) {
  const char *what = "sps_cosine_grad_workspace_size";
  if (!bytes) return set_error(SPS_ERR_INVALID_ARGUMENT, "NULL output pointer");
  if (!other) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL handle", what);
  if (nnz < 0) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: negative size", what);
  if (nnz >= kMax31) return set_error(SPS_ERR_OVERFLOW, "%s: sizes must be below 2^31", what);
  *bytes = other->g.n_sub > 1 ? (size_t)other->g.n_sub * (size_t)nnz * 4 : 0;
  return SPS_OK;
}

sps_status sps_cosine_grad(const sps_csr *rows, const sps_items *other, int32_t chunk,
                           const sps_scores *grad, int32_t transposed, int32_t first, float *du,
                           void *workspace, size_t workspace_bytes, void *stream) {
  const char *what = "sps_cosine_grad";
  sps_status st = check_csr(rows, what);
  if (st != SPS_OK) return st;
  if (!other) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL handle", what);
  if (rows->n_cols != other->dim)
    return set_error(SPS_ERR_DIM_MISMATCH, "%s: dims of the two sides differ: %lld and %lld", what,
                     (long long)rows->n_cols, (long long)other->dim);
  if (chunk < 0 || chunk >= other->g.num_chunks)
    return set_error(SPS_ERR_CHUNK_RANGE, "%s: chunk %d outside [0, %d)", what, chunk,
                     other->g.num_chunks);
  st = sps::check_scores(grad, what);
  if (st != SPS_OK) return st;
  const int64_t n_rows = rows->n_rows;
  const int64_t len = other->g.chunk_end(chunk) - other->g.chunk_begin(chunk);
  const int64_t gr = transposed ? len : n_rows, gc = transposed ? n_rows : len;
  if (grad->n_rows != gr || grad->n_cols != gc)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: the gradient is %lld x %lld, not %lld x %lld",
                     what, (long long)grad->n_rows, (long long)grad->n_cols, (long long)gr,
                     (long long)gc);
  if (n_rows == 0 || rows->nnz == 0) return SPS_OK;
  if (!du) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL output", what);
  sps::WalkArgs a{};
  a.indptr = rows->indptr;
  a.indices = rows->indices;
  a.nnz = rows->nnz;
  a.n_rows = n_rows;
  a.n_groups = (n_rows + sps::kGradRows - 1) / sps::kGradRows;
  a.g = other->g;
  a.chunk = chunk;
  a.dinfo = other->dinfo;
  a.dtab = other->dtab;
  a.post = other->post;
  a.slice_base = other->slice_base;
  a.grad = grad->data;
  a.ld = grad->ld;
  a.transposed = transposed != 0;
  a.first = first != 0;
  a.du = du;
  if (other->g.n_sub > 1) {
    if (!workspace) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL workspace", what);
    if (reinterpret_cast<uintptr_t>(workspace) & 15)
      return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: workspace must be 16-byte aligned", what);
    const size_t all = (size_t)other->g.n_sub * (size_t)rows->nnz * 4;
    if (workspace_bytes < all)
      return set_error(SPS_ERR_WORKSPACE_TOO_SMALL, "%s: need %zu bytes, got %zu", what, all,
                       workspace_bytes);
    a.parts = static_cast<float *>(workspace);
  }
  const int64_t blocks = a.n_groups * other->g.n_sub;
  st = sps::check_grid(blocks, sps::kGradThreads, what);
  if (st != SPS_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((uint32_t)blocks), block(sps::kGradThreads);
  if (grad->dtype == SPS_F32)
    hipLaunchKernelGGL((sps::grad_walk_kernel<float>), grid, block, 0, s, a);
  else if (grad->dtype == SPS_F16)
    hipLaunchKernelGGL((sps::grad_walk_kernel<sps::f16_t>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((sps::grad_walk_kernel<sps::bf16_t>), grid, block, 0, s, a);
  if (a.parts) {
    int64_t fold = (rows->nnz + 255) / 256;
    if (fold > 2048) fold = 2048;
    hipLaunchKernelGGL(sps::grad_fold_kernel, dim3((uint32_t)fold), dim3(256), 0, s, a);
  }
  return sps::launch_status(what);
}

sps_status sps_cosine_grad_values(const sps_csr *rows, const float *du, float *dv, void *stream) {
  const char *what = "sps_cosine_grad_values";
  const sps_status st = check_csr(rows, what);
  if (st != SPS_OK) return st;
  if (rows->n_rows == 0 || rows->nnz == 0) return SPS_OK;
  if (!du || !dv) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL gradient", what);
  const sps_status fits = sps::check_grid((rows->n_rows + 3) / 4, 256, what);
  if (fits != SPS_OK) return fits;
  hipLaunchKernelGGL(sps::grad_values_kernel, dim3((uint32_t)((rows->n_rows + 3) / 4)), dim3(256),
                     0, reinterpret_cast<hipStream_t>(stream), rows->n_rows, rows->nnz,
                     rows->indptr, rows->values, du, dv);
  return sps::launch_status(what);
}

sps_status sps_cosine_grad_both_workspace_size(int64_t nnz_queries, int64_t nnz_items,
                                               size_t *bytes) {
  if (!bytes) return set_error(SPS_ERR_INVALID_ARGUMENT, "NULL output pointer");
  if (nnz_queries < 0 || nnz_items < 0)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "negative size");
  // places are 32-bit, and a wave looks up to 512 past one
  const int64_t most = kMax31 - 65536;
  if (nnz_queries >= most || nnz_items >= most || nnz_queries + nnz_items >= most)
    return set_error(SPS_ERR_OVERFLOW, "entries of both sides must be below 2^31 - 2^16");
  *bytes = both_layout(nnz_queries + nnz_items).total;
  return SPS_OK;
}

sps_status sps_cosine_grad_both(const sps_csr *queries, const sps_csr *items,
                                const sps_scores *grad, float *grad_queries, float *grad_items,
                                void *workspace, size_t workspace_bytes, void *stream) {
  const char *what = "sps_cosine_grad_both";
  sps_status st = check_csr(queries, what);
  if (st == SPS_OK) st = check_csr(items, what);
  if (st == SPS_OK) st = sps::check_scores(grad, what);
  if (st != SPS_OK) return st;
  if (queries->n_cols != items->n_cols)
    return set_error(SPS_ERR_DIM_MISMATCH, "%s: dims of the two sides differ: %lld and %lld", what,
                     (long long)queries->n_cols, (long long)items->n_cols);
  if (grad->n_rows != queries->n_rows || grad->n_cols != items->n_rows)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: the gradient is not %lld x %lld", what,
                     (long long)queries->n_rows, (long long)items->n_rows);
  size_t need = 0;
  st = sps_cosine_grad_both_workspace_size(queries->nnz, items->nnz, &need);
  if (st != SPS_OK) return st;
  if ((queries->nnz > 0 && !grad_queries) || (items->nnz > 0 && !grad_items))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL output", what);
  const int64_t n = queries->nnz + items->nnz;
  if (n == 0) return SPS_OK;
  if (!workspace) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL workspace", what);
  if (workspace_bytes < need)
    return set_error(SPS_ERR_WORKSPACE_TOO_SMALL, "%s: need %zu bytes, got %zu", what, need,
                     workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", what);
  const BothLayout L = both_layout(n);
  char *b = static_cast<char *>(workspace);
  sps::BothArgs a{};
  a.unit = reinterpret_cast<float *>(b + L.unit);
  a.row = reinterpret_cast<int32_t *>(b + L.row);
  for (int i = 0; i < 2; ++i) {
    a.key[i] = reinterpret_cast<int32_t *>(b + L.key[i]);
    a.load[i] = reinterpret_cast<uint2 *>(b + L.load[i]);
  }
  a.hist = reinterpret_cast<int32_t *>(b + L.hist);
  a.total = reinterpret_cast<int32_t *>(b + L.sums);
  a.per_block = L.per_block;
  int bits = 1;
  while (bits < 31 && (queries->n_cols - 1) >> bits) ++bits;
  a.passes = (bits + sps::kMaxBits - 1) / sps::kMaxBits;
  a.bits = (bits + a.passes - 1) / a.passes;
  if (a.bits < 2) a.bits = 2;  // histograms are read four bins at a time
  a.last = (a.passes - 1) & 1;
  a.grad = grad->data;
  a.ld = grad->ld;
  const sps_csr *m[2] = {queries, items};
  float *dv[2] = {grad_queries, grad_items};
  int64_t base = 0, groups = 0;
  int32_t blocks = 0;
  for (int i = 0; i < 2; ++i) {
    sps::BothSide &s = a.s[i];
    s.indptr = m[i]->indptr;
    s.indices = m[i]->indices;
    s.values = m[i]->values;
    s.dv = dv[i];
    s.n_rows = m[i]->n_rows;
    s.nnz = m[i]->nnz;
    s.base = base;
    base += s.nnz;
    s.block0 = blocks;
    s.blocks = (int32_t)((s.nnz + a.per_block - 1) / a.per_block);
    blocks += s.blocks;
    s.slots = slots_of(s.nnz);
    s.lists = reinterpret_cast<uint4 *>(b + L.lists) + (i ? a.s[0].slots : 0);
    s.groups = (s.n_rows + sps::kWalkRows - 1) / sps::kWalkRows;
    groups = (groups + 7) / 8 * 8 + s.groups;
  }
  const int64_t rows = queries->n_rows + items->n_rows;
  const int64_t slots = (int64_t)a.s[0].slots + a.s[1].slots;
  const int64_t unit_blocks =
      blocks + (rows + sps::kSortWaves - 1) / sps::kSortWaves +
      (slots + sps::kSortThreads * sps::kFillEach - 1) / (sps::kSortThreads * sps::kFillEach);
  st = sps::check_grid(groups, sps::kWalkThreads, what);
  if (st == SPS_OK) st = sps::check_grid(unit_blocks, sps::kSortThreads, what);
  if (st != SPS_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 sort(sps::kSortThreads);
  hipLaunchKernelGGL(sps::both_unit_kernel, dim3((uint32_t)unit_blocks), sort, 0, s, a);
  for (a.pass = 0; a.pass < a.passes; ++a.pass) {
    if (a.pass > 0)
      hipLaunchKernelGGL(sps::both_hist_kernel, dim3((uint32_t)blocks), sort, 0, s, a);
    hipLaunchKernelGGL(sps::both_prefix_kernel, dim3(2u * (uint32_t)(((1 << a.bits) + 63) / 64)),
                       dim3(sps::kPrefixWaves * 64), 0, s, a);
    hipLaunchKernelGGL(sps::both_scatter_kernel, dim3((uint32_t)blocks), sort, 0, s, a);
  }
  hipLaunchKernelGGL(sps::both_lists_kernel, dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, s, a);
  const dim3 grid((uint32_t)groups), block(sps::kWalkThreads);
  if (grad->dtype == SPS_F32)
    hipLaunchKernelGGL((sps::both_walk_kernel<float>), grid, block, 0, s, a);
  else if (grad->dtype == SPS_F16)
    hipLaunchKernelGGL((sps::both_walk_kernel<sps::f16_t>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((sps::both_walk_kernel<sps::bf16_t>), grid, block, 0, s, a);
  return sps::launch_status(what);
}

}  // extern "C"
