// sps_rows.h -- shared by the kernels that read rows of scores (selection,
// distillation): element types, 16-byte loads and block reductions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sps.h"
#include "sps_device.h"
#include "sps_internal.h"

namespace sps {

struct f16_t { uint16_t u; };
struct bf16_t { uint16_t u; };

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(f16_t x) { return (float)__builtin_bit_cast(_Float16, x.u); }
__device__ __forceinline__ float to_f32(bf16_t x) {
  return __builtin_bit_cast(float, (uint32_t)x.u << 16);
}
// one rounding to the nearest, ties to even
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ f16_t from_f32<f16_t>(float x) {
  return {__builtin_bit_cast(uint16_t, (_Float16)x)};
}
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float x) {
  return {__builtin_bit_cast(uint16_t, (__bf16)x)};
}

// Elements of one 16-byte vector. Rows start at any multiple of the element
// size, so the vector type claims no more alignment than an element has.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Vec {
  T e[kVec<T>];
};

// float -> uint32 whose unsigned order is the order of the floats; 0 for what
// is no candidate (NaN and -inf). Both zeros give one value.
__device__ __forceinline__ uint32_t order_bits(float f) {
  const float g = f + 0.0f;
  const int32_t b = __builtin_bit_cast(int32_t, g);
  const uint32_t u = (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
  return g > -__builtin_inff() ? u : 0u;
}
__device__ __forceinline__ float unorder_bits(uint32_t u) {
  return __builtin_bit_cast(float, (u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}

inline int32_t dtype_size(int32_t dtype) { return dtype == SPS_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) { return dtype >= SPS_F32 && dtype <= SPS_BF16; }

// The checks that every call on a view of scores shares.
inline sps_status check_scores(const sps_scores *s, const char *what) {
  if (!s) return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL scores", what);
  if (!dtype_ok(s->dtype))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: unknown element type %d", what, s->dtype);
  if (s->n_rows < 0 || s->n_cols < 0 || s->col_begin < 0)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: negative size", what);
  const int64_t max31 = 2147483647ll;
  if (s->n_rows >= max31 || s->n_cols >= max31 || s->col_begin >= max31 ||
      s->col_begin + s->n_cols >= max31)
    return set_error(SPS_ERR_OVERFLOW, "%s: rows and columns must be below 2^31", what);
  if (s->ld < s->n_cols)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: ld %lld below the %lld columns", what,
                     (long long)s->ld, (long long)s->n_cols);
  if (s->n_rows > 0 && (uint64_t)s->ld > (uint64_t)INT64_MAX / 4 / (uint64_t)s->n_rows)
    return set_error(SPS_ERR_OVERFLOW, "%s: n_rows * ld overflows", what);
  if (s->n_rows > 0 && s->n_cols > 0 && !s->data)
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: NULL data", what);
  if (reinterpret_cast<uintptr_t>(s->data) % (uintptr_t)dtype_size(s->dtype))
    return set_error(SPS_ERR_INVALID_ARGUMENT, "%s: data not aligned to its elements", what);
  return SPS_OK;
}

// Whether two sets of rows (n rows of `bytes` bytes, `stride` bytes apart) share a byte: rows may
// lie between each other's, as the halves of one wide buffer do.
struct RowBytes {
  const void *at;
  int64_t n, bytes, stride;
};
inline bool rows_overlap(RowBytes a, RowBytes b) {
  if (a.n == 0 || b.n == 0 || a.bytes == 0 || b.bytes == 0) return false;
  if (a.n > b.n) {
    const RowBytes x = a;
    a = b;
    b = x;
  }
  const __int128 a0 = reinterpret_cast<uintptr_t>(a.at), b0 = reinterpret_cast<uintptr_t>(b.at);
  const __int128 a1 = a0 + (__int128)(a.n - 1) * a.stride + a.bytes;
  const __int128 b1 = b0 + (__int128)(b.n - 1) * b.stride + b.bytes;
  if (a1 <= b0 || b1 <= a0) return false;
  if (b.n == 1) return true;
  // row j of b starts d + j b.stride bytes behind a row of a; they share a byte where that is
  // above -b.bytes and below a.bytes. With equal strides rows i and j stand as 0 and j - i do
  const auto floor_div = [](__int128 x, __int128 y) { return x / y - (x % y < 0); };
  const auto meets = [&](__int128 d, __int128 first) {
    const __int128 least = floor_div(-b.bytes - d, b.stride) + 1;
    const __int128 most = floor_div(a.bytes - 1 - d, b.stride);
    return (least > first ? least : first) <= (most < b.n - 1 ? most : b.n - 1);
  };
  if (a.stride == b.stride) return meets(b0 - a0, 1 - a.n);
  // ranges that meet at different strides: rare, and a launch's rows are at most 2^24
  for (int64_t i = 0; i < a.n; ++i)
    if (meets(b0 - a0 - (__int128)i * a.stride, 0)) return true;
  return false;
}

// A launch's threads are counted in 32 bits.
inline sps_status check_grid(int64_t blocks, int64_t threads, const char *what) {
  if (blocks > 4294967295ll / threads)
    return set_error(SPS_ERR_OVERFLOW, "%s: too many rows for a launch", what);
  return SPS_OK;
}

inline sps_status launch_status(const char *what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(SPS_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return SPS_OK;
}

}  // namespace sps
