// sps_gemm.h -- the tiled matrix product of the operators on dense rows.
//
// D[r][c] = sum over k of Q[r][k] P[c][k]: both operands have their k in one
// run of bytes a row, which is how rows of embeddings lie. Everything here
// counts in bytes: a step takes 128 bytes of k of every row (64 values of 16
// bits, 128 of 8), a matrix instruction 64 of them, 16 bytes a lane, whatever
// the type, so one body serves bf16, fp16 and int8.
//
// Tile: TC columns by TR rows of D a workgroup, WC x WR waves. P is the matrix
// instructions' first operand, so a lane holds four neighbouring columns of
// one row: rows of D are stored, reduced and scaled without a move between
// lanes. Tiles of both operands go straight from memory to LDS (no registers,
// no ds_write), two buffers deep: the next step's loads are issued behind the
// barrier that frees their buffer and have a whole step to arrive.
//
// LDS: a row's 128 bytes in eight 16-byte places, chunk c at place c ^ (row &
// 7): a direct load fills 64 lanes' places in order, so the permutation is
// applied to the addresses loaded from; the reads of 16 rows then meet every
// bank equally.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sps_rows.h"

namespace sps {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct OpF16 {
  using Frag = f16x8;
  using Acc = f32x4;
  static __device__ __forceinline__ Acc mma(Frag p, Frag q, Acc a) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(p, q, a, 0, 0, 0);
  }
};
struct OpBf16 {
  using Frag = bf16x8;
  using Acc = f32x4;
  static __device__ __forceinline__ Acc mma(Frag p, Frag q, Acc a) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q, a, 0, 0, 0);
  }
};
struct OpI8 {
  using Frag = i32x4;
  using Acc = i32x4;
  static __device__ __forceinline__ Acc mma(Frag p, Frag q, Acc a) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(p, q, a, 0, 0, 0);
  }
};

// Rows of an operand: `rows` rows, ld bytes apart, base and ld on 16-byte
// boundaries. A float32 matrix stands in three planes of bf16 (a value's
// leading, middle and last 8 bits), `plane` bytes apart.
struct GemmOperand {
  const uint8_t *base;
  int64_t rows;
  int64_t ld;
  int64_t plane;
};

// k_bytes of every row take part (a multiple of 16). With planes != 0 the six
// products of planes that reach 2^-24 of a product are summed one after
// another, as if k were six times as long. splits > 1: workgroup (tile, z)
// sums the z-th part of the steps.
struct GemmArgs {
  GemmOperand q, p;
  int64_t k_bytes;
  int32_t planes;
  int32_t splits;
  int32_t tiles_c, tiles_r;
};

constexpr int kStep = 128;                    // bytes of k a step
constexpr uint32_t kMostBytes = 0x7fffffffu;  // of a tile's rows: offsets are 32 bits
constexpr int kSegments = 6;

// planes of a float32 product's six parts: hi hi, hi mid, mid hi, hi low, low hi, mid mid
__device__ __forceinline__ int seg_q(int s) { return (0x001021 >> (4 * (5 - s))) & 15; }
__device__ __forceinline__ int seg_p(int s) { return (0x010201 >> (4 * (5 - s))) & 15; }

// Workgroups go to the 8 XCDs in turn; each XCD has an L2 of its own. A run of
// neighbouring tiles goes to one XCD, and within it kGroup rows of tiles are
// walked together, so that both operands' tiles are met again while they are
// still in that L2.
constexpr int kXcds = 8;
constexpr int kGroup = 4;
__device__ __forceinline__ void tile_of(uint32_t id, int32_t tiles_c, int32_t tiles_r, int *tc,
                                        int *tr) {
  const uint32_t all = (uint32_t)tiles_c * (uint32_t)tiles_r;
  const uint32_t x = id % kXcds, at = id / kXcds;
  const uint32_t each = all / kXcds, more = all % kXcds;
  const uint32_t t = x * each + (x < more ? x : more) + at;
  const uint32_t per = kGroup * (uint32_t)tiles_c;
  const uint32_t g = t / per, in = t % per;
  const uint32_t first = g * kGroup;
  const uint32_t h = (uint32_t)tiles_r - first < kGroup ? (uint32_t)tiles_r - first : kGroup;
  *tr = (int)(first + in % h);
  *tc = (int)(in / h);
}

typedef __attribute__((address_space(3))) uint8_t lds_u8;

template <class Op, int TC, int TR, int WC, int WR>
struct GemmTile {
  static constexpr int kThreads = 64 * WC * WR;
  static constexpr int kC = TC, kR = TR;
  static constexpr int kFragC = TC / WC / 16, kFragR = TR / WR / 16;
  static constexpr int kBuf = (TC + TR) * kStep;  // bytes of one step
  static constexpr int kRowsLoad = 8 * WC * WR;   // rows that one load of every wave fills
  static constexpr int kLoadsP = TC / kRowsLoad, kLoadsQ = TR / kRowsLoad;
  static_assert(TC % kRowsLoad == 0 && TR % kRowsLoad == 0, "whole loads");
  static_assert(2 * kBuf <= 160 * 1024, "LDS");
  using Acc = typename Op::Acc;
  using Frag = typename Op::Frag;

  Acc acc[kFragC][kFragR];

  // The sum over steps [begin, end) for the tile at (row0, col0).
  __device__ __forceinline__ void run(const GemmArgs &a, int64_t row0, int64_t col0, int begin,
                                      int end, uint8_t *lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wc = wave % WC, wr = wave / WC;
#pragma unroll
    for (int i = 0; i < kFragC; ++i)
#pragma unroll
      for (int j = 0; j < kFragR; ++j) acc[i][j] = Acc{};
    if (begin >= end) return;

    const int steps = (int)((a.k_bytes + kStep - 1) / kStep);  // of one segment
    const uint32_t ld_p = (uint32_t)a.p.ld, ld_q = (uint32_t)a.q.ld;
    const auto left = [](int64_t rows, int64_t first, int64_t ld) {
      const int64_t b = (rows - first) * ld;  // rows past the last read as zeros
      return (uint32_t)(b < (int64_t)kMostBytes ? b : (int64_t)kMostBytes);
    };
    const uint32_t size_p = left(a.p.rows, col0, a.p.ld), size_q = left(a.q.rows, row0, a.q.ld);
    const uint8_t *base_p = a.p.base + col0 * a.p.ld, *base_q = a.q.base + row0 * a.q.ld;

    // this lane's place in a load: row lane / 8 of the wave's eight, and the chunk that belongs there
    const uint32_t row = (uint32_t)(wave * 8 + (lane >> 3));
    const uint32_t chunk = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
    const uint32_t off_p = row * ld_p + chunk, off_q = row * ld_q + chunk;
    uint8_t *const to = lds + wave * 1024;

    auto load = [&](int step) {
      const int seg = a.planes ? step / steps : 0;
      const uint32_t k = (uint32_t)(step - seg * steps) * kStep;
      const auto rp = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t *>(base_p + (a.planes ? seg_p(seg) * a.p.plane : 0)), 0, (int)size_p,
          0x00020000);
      const auto rq = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t *>(base_q + (a.planes ? seg_q(seg) * a.q.plane : 0)), 0, (int)size_q,
          0x00020000);
      // past the end of k: an offset past the buffer's, which reads zeros
      const bool in = (int64_t)k + chunk < a.k_bytes;
      const uint32_t at_p = in ? off_p + k : 0x80000000u, at_q = in ? off_q + k : 0x80000000u;
      uint8_t *const b = to + (step & 1) * kBuf;
#pragma unroll
      for (int i = 0; i < kLoadsP; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (lds_u8 *)(b + i * kRowsLoad * kStep), 16,
                                                 (int)(at_p + (uint32_t)i * kRowsLoad * ld_p), 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kLoadsQ; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (lds_u8 *)(b + (TC + i * kRowsLoad) * kStep), 16,
                                                 (int)(at_q + (uint32_t)i * kRowsLoad * ld_q), 0, 0, 0);
    };

    // a fragment: row lane % 16, bytes 16 (lane / 16) of 64; the other 64 bytes are places ^ 4
    const int in_row = (lane & 15) * kStep;
    const int at0 = in_row + (((lane >> 4) ^ (lane & 7)) * 16), at1 = at0 ^ 64;
    const int from_p = wc * (kFragC * 16) * kStep, from_q = (TC + wr * (kFragR * 16)) * kStep;

    load(begin);
    for (int s = begin; s < end; ++s) {
      // every wave's loads of step s are in LDS, and its reads of the other buffer are done
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (s + 1 < end) load(s + 1);
      __builtin_amdgcn_sched_barrier(0);
      const uint8_t *const b = lds + (s & 1) * kBuf;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int at = half ? at1 : at0;
        Frag p[kFragC], q[kFragR];
#pragma unroll
        for (int i = 0; i < kFragC; ++i)
          p[i] = *reinterpret_cast<const Frag *>(b + from_p + i * 16 * kStep + at);
#pragma unroll
        for (int j = 0; j < kFragR; ++j)
          q[j] = *reinterpret_cast<const Frag *>(b + from_q + j * 16 * kStep + at);
#pragma unroll
        for (int i = 0; i < kFragC; ++i)
#pragma unroll
          for (int j = 0; j < kFragR; ++j) acc[i][j] = Op::mma(p[i], q[j], acc[i][j]);
      }
    }
    // the buffers may be used again by what follows
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  // Place of acc[i][j][e] in the tile: row_of(j), col_of(i) + e.
  __device__ __forceinline__ int row_of(int j) const {
    const int wave = threadIdx.x >> 6;
    return (wave / WC) * (kFragR * 16) + j * 16 + (threadIdx.x & 15);
  }
  __device__ __forceinline__ int col_of(int i) const {
    const int wave = threadIdx.x >> 6;
    return (wave % WC) * (kFragC * 16) + i * 16 + ((threadIdx.x & 63) >> 4) * 4;
  }
};

// The tile, its rows and columns and its part of the steps.
struct GemmPlace {
  int64_t row0, col0;
  int begin, end;
  int32_t z;
};
template <int TC, int TR>
__device__ __forceinline__ GemmPlace gemm_place(const GemmArgs &a) {
  GemmPlace g;
  int tc, tr;
  const uint32_t tiles = (uint32_t)a.tiles_c * (uint32_t)a.tiles_r;
  g.z = (int32_t)(blockIdx.x / tiles);
  tile_of(blockIdx.x % tiles, a.tiles_c, a.tiles_r, &tc, &tr);
  g.row0 = (int64_t)tr * TR;
  g.col0 = (int64_t)tc * TC;
  const int steps = (int)((a.k_bytes + kStep - 1) / kStep) * (a.planes ? kSegments : 1);
  g.begin = (int)((int64_t)steps * g.z / a.splits);
  g.end = (int)((int64_t)steps * (g.z + 1) / a.splits);
  return g;
}

template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Four {
  T e[4];
};

// Four neighbouring values of a row.
template <typename T>
__device__ __forceinline__ void put_four(T *out, int64_t col, int64_t cols, const float v[4]) {
  if (col + 4 <= cols) {
    Four<T> t;
#pragma unroll
    for (int e = 0; e < 4; ++e) t.e[e] = from_f32<T>(v[e]);
    *reinterpret_cast<Four<T> *>(out + col) = t;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < cols) out[col + e] = from_f32<T>(v[e]);
  }
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace sps
