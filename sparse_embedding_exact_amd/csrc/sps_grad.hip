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
// Layout. A workgroup keeps kGradRows rows of G over one slice (at most 1024
// items) in LDS and walks the lists of those rows' dims in that slice; every
// entry of a row gets one float32 sum a slice, in a fixed order, and a second
// pass adds the slices. G is read once; the lists come from the L2 of the XCD
// that works on the slice, since consecutive workgroups of an XCD take
// consecutive row groups of the same slice.
#include "sps_rows.h"

namespace sps {

constexpr int kGradRows = 8;      // rows of a workgroup: 8 x 1028 floats are 33 KB of LDS
constexpr int kGradThreads = 256;
constexpr int kGradPitch = kSliceMax + 4;  // rows start 4 banks apart
constexpr int kGradShort = 8;     // a list of at most this many postings is one lane's

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
      if (n <= kGradShort)
        for (int i = 0; i < n; ++i) {
          const uint2 p = post[start + i];
          acc += g[p.x & (kSliceMax - 1)] * __builtin_bit_cast(float, p.y);
        }
      uint64_t rest = __ballot(n > kGradShort);
      while (rest) {
        const int l = __builtin_ctzll(rest);
        rest &= rest - 1;
        const int32_t s = __builtin_amdgcn_readlane(start, l);
        const int32_t m = __builtin_amdgcn_readlane(n, l);
        float part = 0;
        for (int i = lane; i < m; i += 64) {
          const uint2 p = post[s + i];
          part += g[p.x & (kSliceMax - 1)] * __builtin_bit_cast(float, p.y);
        }
        part = wave_sum(part);
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

// One wave a row.
__global__ __launch_bounds__(256) void grad_values_kernel(int64_t n_rows, int64_t nnz,
                                                          const int32_t *__restrict__ indptr,
                                                          const float *__restrict__ values,
                                                          const float *du, float *dv) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= n_rows) return;  // uniform per wave
  const int64_t e0 = clamp64(indptr[row], 0, nnz), e1 = clamp64(indptr[row + 1], e0, nnz);
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
  if (blocks > kMax31)
    return set_error(SPS_ERR_OVERFLOW, "%s: too many rows and slices for a launch", what);
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
  hipLaunchKernelGGL(sps::grad_values_kernel, dim3((uint32_t)((rows->n_rows + 3) / 4)), dim3(256),
                     0, reinterpret_cast<hipStream_t>(stream), rows->n_rows, rows->nnz,
                     rows->indptr, rows->values, du, dv);
  return sps::launch_status(what);
}

}  // extern "C"
