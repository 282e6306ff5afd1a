// sps_gemm.h -- the tiled matrix product of the operators on dense rows.
//
// D[r][c] = sum over k of Q[r][k] P[c][k]: both operands have their k in one
// run of bytes a row, which is how rows of embeddings lie. Everything here
// counts in bytes: a step takes 128 bytes of k of every row (64 values of 16
// bits, 128 of 8), a matrix instruction 64 of them, 16 bytes a lane, whatever
// the type, so one body serves bf16, fp16 and int8.
//
// Or Q stands turned, Q[k][r] with a run of r a row of k (16-bit values): its
// tile is then 64 rows of k, read through the transposing LDS load.
//
// Tile: TC columns by TR rows of D a workgroup, WC x WR waves. P is the matrix
// instructions' first operand, so a lane holds four neighbouring columns of
// one row: rows of D are stored, reduced and scaled without a move between
// lanes. Tiles of both operands go straight from memory to LDS (no registers,
// no ds_write), two buffers deep: the next step's loads are issued behind the
// barrier that frees their buffer and have a whole step to arrive. A workgroup
// goes from tile to tile, and the next one's first two steps are loaded while
// this one's sums are put away.
//
// What bounds it: bf16 tiles of 256 x 256 reach 1.2 PFLOP/s on random values and
// 1.55 on zeros, without their loads 1.16 and 1.51 (the library's product of
// 8192^3 1.26 to 1.47): the power that the matrix instructions draw, then, where
// k is short, what becomes of a tile's sums while its CU multiplies nothing (4
// to 8 us a tile: 65,536 exponentials, or scores scaled, and their stores).
// 32 x 32 x 16 instructions: 1118 against 1190 TFLOP/s; four waves of 128 x 128
// spill (300 against 218 us for 4095 x 30,522 x 768 of logits).
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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct OpF16 {
  using Type = f16_t;
  static constexpr int kPlanes = 1;
  using Frag = f16x8;
  using Acc = f32x4;
  static __device__ __forceinline__ Acc mma(Frag p, Frag q, Acc a) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(p, q, a, 0, 0, 0);
  }
};
struct OpBf16 {
  using Type = bf16_t;
  static constexpr int kPlanes = 1;
  using Frag = bf16x8;
  using Acc = f32x4;
  static __device__ __forceinline__ Acc mma(Frag p, Frag q, Acc a) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q, a, 0, 0, 0);
  }
};
struct OpI8 {
  static constexpr int kPlanes = 1;
  using Frag = i32x4;
  using Acc = i32x4;
  static __device__ __forceinline__ Acc mma(Frag p, Frag q, Acc a) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(p, q, a, 0, 0, 0);
  }
};

// float32 as two planes of fp16
struct OpF32 : OpF16 {
  using Type = float;
  static constexpr int kPlanes = 2;
};

// Rows of an operand: `rows` rows, ld bytes apart, base and ld on 16-byte
// boundaries. A float32 matrix stands, scaled, in two planes of fp16 (a value's
// leading 11 bits, and 11 of what is left), `plane` bytes apart.
struct GemmOperand {
  const uint8_t *base;
  int64_t rows;
  int64_t ld;
  int64_t plane;
};

// k_bytes of every row take part (a multiple of 16). With planes their three
// products but that of both rests (2^-22 of a product) are summed one after
// another, as if k were three times as long. The first main_r rows of tiles are
// summed whole; of the tail_r behind them part z of `splits` takes the z-th
// part of the steps.
struct GemmArgs {
  GemmOperand q, p;
  int64_t k_bytes;
  int64_t k_rows;  // of a turned q
  int32_t tiles_c, main_r, tail_r, splits;
};

constexpr int kStep = 128;                    // bytes of k a step
constexpr uint32_t kMostBytes = 0x7fffffffu;  // of a tile's rows: offsets are 32 bits
constexpr int kSegments = 3;

// planes of a float32 product's parts: lead lead, lead rest, rest lead
__device__ __forceinline__ int seg_q(int s) { return s == 2; }
__device__ __forceinline__ int seg_p(int s) { return s == 1; }

// Workgroups go to the 8 XCDs in turn; each XCD has an L2 of its own. A run of
// neighbouring tiles goes to one XCD, and within it kGroup rows of tiles are
// walked together, so that both operands' tiles are met again while they are
// still in that L2. Cross entropy of 2000 x 8192 x 768 138 us, in plain order
// 151; logits of 4095 x 30,522 x 768 190, plain 199, kGroup 1 199, 16 195; 8-bit
// scores 2000 x 8192 23.4 us, kGroup 1 26.4.
constexpr int kXcds = 8;
constexpr int kGroup = 4;
__device__ __forceinline__ uint32_t in_xcd_order(uint32_t id, uint32_t all) {
  const uint32_t x = id % kXcds, each = all / kXcds, more = all % kXcds;
  return x * each + (x < more ? x : more) + id / kXcds;
}
__device__ __forceinline__ void tile_of(uint32_t t, int32_t tiles_c, int32_t tiles_r, int *tc, int *tr) {
  const uint32_t per = kGroup * (uint32_t)tiles_c;
  const uint32_t g = t / per, in = t % per;
  const uint32_t first = g * kGroup;
  const uint32_t h = (uint32_t)tiles_r - first < kGroup ? (uint32_t)tiles_r - first : kGroup;
  *tr = (int)(first + in % h);
  *tc = (int)(in / h);
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

// Four values in a type's bits, side by side.
template <typename T>
struct QuadOf {
  typedef uint32_t Bits __attribute__((ext_vector_type(sizeof(T))));
};
template <typename T>
__device__ __forceinline__ typename QuadOf<T>::Bits quad_of(const float v[4]) {
  struct {
    T e[4];
  } q = {{from_f32<T>(v[0]), from_f32<T>(v[1]), from_f32<T>(v[2]), from_f32<T>(v[3])}};
  return __builtin_bit_cast(typename QuadOf<T>::Bits, q);
}

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// A tile's rows and columns and its part of the steps (z < 0: all of them).
struct GemmPlace {
  int64_t row0, col0;
  int begin, end;
  int32_t z;
};
template <class Op, int TC, int TR>
__device__ __forceinline__ GemmPlace gemm_place(const GemmArgs &a, uint32_t id) {
  GemmPlace g;
  int tc, tr;
  const int steps = (int)((a.k_bytes + kStep - 1) / kStep) * (Op::kPlanes > 1 ? kSegments : 1);
  const uint32_t main = (uint32_t)a.tiles_c * (uint32_t)a.main_r;
  if (id < main) {
    g.z = -1;
    tile_of(in_xcd_order(id, main), a.tiles_c, a.main_r, &tc, &tr);
    g.begin = 0;
    g.end = steps;
  } else {
    const uint32_t tail = (uint32_t)a.tiles_c * (uint32_t)a.tail_r;
    id = in_xcd_order(id - main, tail * (uint32_t)a.splits);
    g.z = (int32_t)(id / tail);
    tile_of(id % tail, a.tiles_c, a.tail_r, &tc, &tr);
    tr += a.main_r;
    g.begin = (int)((int64_t)steps * g.z / a.splits);
    g.end = (int)((int64_t)steps * (g.z + 1) / a.splits);
  }
  g.row0 = (int64_t)tr * TR;
  g.col0 = (int64_t)tc * TC;
  return g;
}

template <class Op, int TC, int TR, int WC, int WR, bool QT = false>
struct GemmTile {
  static constexpr int kThreads = 64 * WC * WR;
  static constexpr int kC = TC, kR = TR;
  static constexpr int kFragC = TC / WC / 16, kFragR = TR / WR / 16;
  static constexpr int kBuf = (TC + TR) * kStep;  // bytes of one step
  static constexpr int kWaveLds = 4096;           // a wave's part for what it stores
  static constexpr int kLds = 2 * kBuf + kWaveLds * WC * WR;
  static constexpr int kRowsLoad = 8 * WC * WR;   // rows that one load of every wave fills
  static constexpr int kLoadsP = TC / kRowsLoad, kLoadsQ = TR / kRowsLoad;
  static constexpr int kLoads = kLoadsP + kLoadsQ;
  static_assert(TC % kRowsLoad == 0 && TR % kRowsLoad == 0, "whole loads");
  static_assert(kLds <= 160 * 1024, "LDS");
  using Acc = typename Op::Acc;
  using Frag = typename Op::Frag;

  const GemmArgs &a;
  uint8_t *const lds;
  int lane;
  const int wave, wc, wr;
  const uint32_t ld_p, ld_q, chunk;
  uint32_t off_p, off_q;
  Acc acc[kFragC][kFragR];
  GemmPlace at;  // of the sums
  // of the loads, which are ahead of them
  uint8_t *base_p, *base_q;
  int size_p, size_q, seg;
  int64_t col_q;
  uint32_t k;
  bool any;

  // Turned: 1024 bytes are 1024 / (2 TR) rows of k. A transposing read takes 32 bytes of 16 of
  // them, rows k and k + 8 apart among them: pair p of 16-byte chunks of row k stands at p ^ turn(k),
  // turn(k) = k % 4 + 4 (k / 8 % 2), so that 8 rows meet every bank once.
  static constexpr int kPlaces = TR * 2 / 16;
  static constexpr int kNextQ = QT ? (64 / kPlaces) * WC * WR : kRowsLoad;  // rows between a wave's loads
  static_assert(!QT || kNextQ % 16 == 0, "one turn(k) for all loads of a lane");

  __device__ __forceinline__ GemmTile(const GemmArgs &args, uint8_t *shared)
      : a(args), lds(shared), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), wc(wave % WC),
        wr(wave / WC), ld_p((uint32_t)args.p.ld), ld_q((uint32_t)args.q.ld),
        // this lane's place in a load: row lane / 8 of the wave's eight, and the chunk that belongs there
        chunk((uint32_t)(((lane & 7) ^ (lane >> 3)) * 16)) {
    const uint32_t row = (uint32_t)(wave * 8 + (lane >> 3));
    off_p = row * ld_p + chunk;
    const uint32_t k_row = (uint32_t)(wave * (64 / kPlaces) + lane / kPlaces), q = (uint32_t)(lane % kPlaces);
    const uint32_t turn = (k_row & 3) | (k_row >> 3 & 1) << 2;
    off_q = QT ? k_row * ld_q + (q ^ (turn << 1)) * 16 : row * ld_q + chunk;
  }

  // What is computed from the lane is computed again in each part of a tile: held over the loop of
  // tiles, it would not leave registers for the sums.
  __device__ __forceinline__ void fresh() { asm volatile("" : "+v"(lane)); }

  // ---- loads

  static __device__ __forceinline__ int left(int64_t rows, int64_t first, int64_t ld, int64_t in = 0) {
    const int64_t b = (rows - first) * ld - in;  // rows past the last read as zeros
    return (int)(b < (int64_t)kMostBytes ? b : (int64_t)kMostBytes);
  }
  __device__ __forceinline__ void place_step(int step) {
    seg = 0;
    if constexpr (Op::kPlanes > 1) {
      const int steps = (int)(((uint32_t)a.k_bytes + kStep - 1) / kStep);
      seg = step / steps;
      step -= seg * steps;
    }
    k = (uint32_t)step * kStep;
  }
  // One step of k into a buffer; past the last one as many loads, of nothing.
  __device__ __forceinline__ void load(uint8_t *buf) {
    uint8_t *const b = buf + wave * 1024;
    const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(
        base_p + (Op::kPlanes > 1 ? seg_p(seg) * a.p.plane : 0), 0, size_p, 0x00020000);
    const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
        base_q + (Op::kPlanes > 1 ? seg_q(seg) * a.q.plane : 0) + (QT ? (int64_t)(k / 2) * a.q.ld : 0),
        0, QT ? any ? left(a.k_rows, (int64_t)(k / 2), a.q.ld, col_q) : 0 : size_q, 0x00020000);
    // past the end of k: an offset past the buffer's, which reads zeros
    const bool in = any && k + chunk < (uint32_t)a.k_bytes;
    const uint32_t at_p = in ? off_p + k : 0x80000000u;
    const uint32_t at_q = (QT ? any : in) ? off_q + (QT ? 0u : k) : 0x80000000u;
#pragma unroll
    for (int i = 0; i < kLoadsP; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (lds_u8 *)(b + i * kRowsLoad * kStep), 16,
                                               (int)(at_p + (uint32_t)i * kRowsLoad * ld_p), 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kLoadsQ; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (lds_u8 *)(b + (TC + i * kRowsLoad) * kStep), 16,
                                               (int)(at_q + (uint32_t)i * kNextQ * ld_q), 0, 0, 0);
    k += kStep;
    if (Op::kPlanes > 1 && k >= (uint32_t)a.k_bytes) {
      k = 0;
      ++seg;
    }
  }
  // The first two steps of a tile's.
  __device__ __forceinline__ void prefetch(const GemmPlace &next) {
    base_p = const_cast<uint8_t *>(a.p.base) + next.col0 * a.p.ld;
    base_q = const_cast<uint8_t *>(a.q.base) + (QT ? next.row0 * 2 : next.row0 * a.q.ld);
    size_p = left(a.p.rows, next.col0, a.p.ld);
    size_q = QT ? 0 : left(a.q.rows, next.row0, a.q.ld);
    col_q = next.row0 * 2;
    const int many = next.end - next.begin;
    place_step(next.begin);
    any = true;
    load(lds);
    any = many > 1;
    load(lds + kBuf);
    any = true;
    // nothing that follows goes before these loads: they are counted
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  // ---- sums

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kFragC; ++i)
#pragma unroll
      for (int j = 0; j < kFragR; ++j) acc[i][j] = Acc{};
  }
  // Sums that go on from those in rows of cols values.
  __device__ __forceinline__ void start(const float *before, int64_t rows, int64_t cols) {
    const bool whole = full();
#pragma unroll
    for (int j = 0; j < kFragR; ++j) {
      const int64_t r = at.row0 + row_of(j);
#pragma unroll
      for (int i = 0; i < kFragC; ++i) {
        const int64_t c = at.col0 + col_of(i);
        const float *const x = before + r * cols + c;
        if (whole) {
          const Four<float> f = *reinterpret_cast<const Four<float> *>(x);
          acc[i][j] = Acc{f.e[0], f.e[1], f.e[2], f.e[3]};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = r < rows && c + e < cols ? x[e] : 0.0f;
        }
      }
    }
  }

  // All but the latest N of this wave's memory operations and its reads of LDS are done, and behind
  // the barrier every wave's.
  template <int N>
  static __device__ __forceinline__ void wait() {
    static_assert(N < 64, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  }
  static __device__ __forceinline__ void barrier() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  __device__ __forceinline__ void read_p(const uint8_t *b, bool half, Frag (&p)[kFragC]) const {
    // a fragment: row lane % 16, bytes 16 (lane / 16) of 64; the other 64 bytes are places ^ 4
    const int in = (lane & 15) * kStep + (((lane >> 4) ^ (lane & 7)) * 16);
#pragma unroll
    for (int i = 0; i < kFragC; ++i)
      p[i] = *reinterpret_cast<const Frag *>(b + (wc * kFragC + i) * 16 * kStep + (half ? in ^ 64 : in));
  }
  __device__ __forceinline__ void read_q(const uint8_t *b, bool half, Frag (&q)[kFragR]) const {
    if constexpr (QT) {
      // Four lanes' 8 bytes are 16 columns of a row of k, 16 lanes' four rows, and a lane receives a
      // column of them: rows 8 (lane / 16) to + 3 of 32, and the four behind with a second read. In
      // assembly, since the compiler makes the builtin wait for every load to LDS on its way, also
      // those to the other buffer; the block ends with its own wait.
      static_assert(kFragR == 4, "four fragments a block");
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      const int four = (lane & 15) >> 2, k_at = (lane >> 4) * 8 + four;
      const int turn = four | ((lane >> 4) & 1) << 2;
      s16x4 x[8];
      uint32_t from[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        from[j] = (uint32_t)(uintptr_t)(lds_u8 *)const_cast<uint8_t *>(b) +
                  (uint32_t)(TC * kStep + k_at * TR * 2 + ((wr * kFragR + j) ^ turn) * 32 + (lane & 3) * 8 +
                             (half ? 32 * TR * 2 : 0));
      asm volatile(
          "ds_read_b64_tr_b16 %0, %8\n\t"
          "ds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
          "ds_read_b64_tr_b16 %2, %9\n\t"
          "ds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
          "ds_read_b64_tr_b16 %4, %10\n\t"
          "ds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
          "ds_read_b64_tr_b16 %6, %11\n\t"
          "ds_read_b64_tr_b16 %7, %11 offset:%12\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]),
            "=&v"(x[6]), "=&v"(x[7])
          : "v"(from[0]), "v"(from[1]), "v"(from[2]), "v"(from[3]), "n"(4 * TR * 2)
          : "memory");
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const s16x4 lo = x[2 * j], hi = x[2 * j + 1];
        const s16x8 both = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        q[j] = __builtin_bit_cast(Frag, both);
      }
    } else {
      const int in = (lane & 15) * kStep + (((lane >> 4) ^ (lane & 7)) * 16);
#pragma unroll
      for (int j = 0; j < kFragR; ++j)
        q[j] = *reinterpret_cast<const Frag *>(b + (TC + (wr * kFragR + j) * 16) * kStep +
                                               (half ? in ^ 64 : in));
    }
  }
  // Half a step from registers, while the next half is read into others and, in a step's second
  // half, the step after the next is loaded. No branches: past the end nothing is loaded, and what
  // is read is not used.
  template <bool LOAD>
  __device__ __forceinline__ void half_step(Frag (&p)[kFragC], Frag (&q)[kFragR], uint8_t *freed,
                                            const uint8_t *b, bool half, Frag (&pn)[kFragC],
                                            Frag (&qn)[kFragR]) {
    if (LOAD) load(freed);
    if (!QT) read_q(b, half, qn);
    read_p(b, half, pn);
#pragma unroll
    for (int i = 0; i < kFragC; ++i) {
#pragma unroll
      for (int j = 0; j < kFragR; ++j) acc[i][j] = Op::mma(p[i], q[j], acc[i][j]);
      if (QT && i == kFragC / 2 - 1) {
        __builtin_amdgcn_sched_barrier(0);
        read_q(b, half, qn);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (!QT) {  // the matrix instructions among the reads and loads
      constexpr int kReads = kFragC + kFragR, kEach = kFragC * kFragR / kReads;
#pragma unroll
      for (int i = 0; i < kReads; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (LOAD && i < kLoads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // Adds the sums over the steps of `at`, whose first two are on their way. `counted`: behind
  // their loads this wave has at least STORES memory operations, which need not be done.
  template <int STORES>
  __device__ __forceinline__ void run(bool counted) {
    const int many = at.end - at.begin;
    fresh();
    if (counted) wait<STORES + kLoads>();
    else wait<0>();
    barrier();
    Frag p0[kFragC], q0[kFragR], p1[kFragC], q1[kFragR];
    read_q(lds, false, q0);
    read_p(lds, false, p0);
    __builtin_amdgcn_sched_barrier(0);
    int here = 0;
    for (int s = 0; s < many; ++s) {
      half_step<false>(p0, q0, nullptr, lds + here, true, p1, q1);
      // behind the barrier this step's buffer has been read to the end and is loaded again, and the
      // next step, which had a whole step's time, is in the other
      if (counted && s == 0) wait<STORES>();
      else wait<0>();
      barrier();
      any = s + 2 < many;
      half_step<true>(p1, q1, lds + here, lds + (here ^ kBuf), false, p0, q0);
      here ^= kBuf;
    }
    // the buffers are free: their loads are done, and behind the barrier the reads
    wait<0>();
    barrier();
  }

  // ---- what becomes of them

  // Rows out of the registers' layout (16 rows of four values a lane) into whole runs: up to 16
  // rows at a time go through this wave's own part of LDS, whose 16-byte places are permuted by the
  // row so that every bank is met equally. Stores of 16-byte runs of 16 rows each reached 3.2 TB/s.
  template <typename T>
  static constexpr int kRun = TC / WC * (int)sizeof(T);
  template <typename T>
  static constexpr int kPass = kWaveLds / kRun<T> < 16 ? kWaveLds / kRun<T> : 16;  // rows
  // Stores of a tile whose rows and columns are all there.
  template <typename T>
  static constexpr int kStores = kFragR * 16 * kRun<T> / 1024;
  template <typename T>
  struct __attribute__((packed, aligned(sizeof(T)))) Words {
    uint32_t w[4];
  };
  template <typename T>
  static __device__ __forceinline__ int place(int row, int byte) {
    constexpr int kOf = kRun<T> / 16;  // places of a row: 8, 16 or 32
    static_assert(kOf == 8 || kOf == 16 || kOf == 32, "permutation");
    const int turn = kOf == 8 ? row >> 1 : kOf == 16 ? row : (row & 7) << 1;
    return row * kRun<T> + (((byte >> 4) ^ turn) << 4) + (byte & 15);
  }
  // What other lanes of the wave wrote to LDS is read behind here: a wave's LDS operations stay in
  // their order once the compiler leaves them so.
  static __device__ __forceinline__ void lanes_meet() {
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
  }
  // To LDS in assembly: the compiler would make it wait for the loads to LDS that are on their way.
  static __device__ __forceinline__ void write_lds(const uint8_t *to, u32x2 v) {
    asm volatile("ds_write_b64 %0, %1" ::"v"((uint32_t)(uintptr_t)(lds_u8 *)const_cast<uint8_t *>(to)), "v"(v)
                 : "memory");
  }
  static __device__ __forceinline__ void write_lds(const uint8_t *to, u32x4 v) {
    asm volatile("ds_write_b128 %0, %1" ::"v"((uint32_t)(uintptr_t)(lds_u8 *)const_cast<uint8_t *>(to)), "v"(v)
                 : "memory");
  }
  // Rows 16 j to 16 j + 15 of this wave: v[i] are the bits of this lane's four values of column group
  // i, to `out` (row 0, column 0 of D) of the given rows and columns; FULL: the tile's are all there.
  // Whole lines that nobody reads soon (STREAM) leave L2 as they come: 10,001 x 30,522 float32
  // scores of 333 dims in 268 us, 372 without; lines in parts are better off waiting there for
  // their other parts (3.0 against 2.8 TB/s). Codes of the cross entropy: equal within 1%.
  template <typename T, bool FULL, bool STREAM, typename Bits>
  __device__ __forceinline__ void store(int j, const Bits (&v)[kFragC], T *out, int64_t ld, int64_t rows,
                                        int64_t cols) const {
    static_assert(sizeof(Bits) == 4 * sizeof(T), "four values");
    constexpr int kLanes = kRun<T> / 16, kOnce = 64 / kLanes, V = 16 / (int)sizeof(T);
    const uint8_t *const mine = lds + 2 * kBuf + wave * kWaveLds;
    const int64_t r0 = at.row0 + (wr * kFragR + j) * 16, c0 = at.col0 + wc * (kFragC * 16);
    const int in = lane % kLanes;
    const int64_t c = c0 + in * V;
    T *const to0 = out + (r0 + lane / kLanes) * ld + c;
#pragma unroll
    for (int pass = 0; pass < 16 / kPass<T>; ++pass) {
      const int row = (lane & 15) - pass * kPass<T>;
      if (kPass<T> == 16 || (row >= 0 && row < kPass<T>))
#pragma unroll
        for (int i = 0; i < kFragC; ++i)
          write_lds(mine + place<T>(row, (i * 16 + (lane >> 4) * 4) * (int)sizeof(T)), v[i]);
      lanes_meet();
#pragma unroll
      for (int n = 0; n < kPass<T> / kOnce; ++n) {
        const int from = n * kOnce + lane / kLanes;
        const u32x4 w = *reinterpret_cast<const u32x4 *>(mine + place<T>(from, in * 16));
        T *const to = to0 + (int64_t)(pass * kPass<T> + n * kOnce) * ld;
        const bool there = r0 + pass * kPass<T> + from < rows;
        if (FULL || (there && c + V <= cols)) {
          if constexpr (STREAM) __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(to));
          else *reinterpret_cast<Words<T> *>(to) = {{w[0], w[1], w[2], w[3]}};
        } else if (there) {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (c + e < cols) {
              const uint32_t u = w[e * (int)sizeof(T) / 4];
              if constexpr (sizeof(T) == 4) to[e] = __builtin_bit_cast(T, u);
              else to[e] = __builtin_bit_cast(T, (uint16_t)(u >> (16 * (e & 1))));
            }
        }
      }
      lanes_meet();
    }
  }
  __device__ __forceinline__ bool full() const {
    return at.row0 + TR <= a.q.rows && at.col0 + TC <= a.p.rows;
  }
  // Values of this lane's columns, `beyond` past the last.
  __device__ __forceinline__ void of_columns(const float *x, float beyond, float (&v)[kFragC][4]) const {
    const int64_t cols = a.p.rows;
    if (at.col0 + TC <= cols) {
#pragma unroll
      for (int i = 0; i < kFragC; ++i) {
        const Four<float> f = *reinterpret_cast<const Four<float> *>(x + at.col0 + col_of(i));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = f.e[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kFragC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t c = at.col0 + col_of(i) + e;
          const float f = x[c < cols ? c : cols - 1];
          v[i][e] = c < cols ? f : beyond;
        }
    }
  }

  // Place of acc[i][j][e] in the tile: row_of(j), col_of(i) + e.
  __device__ __forceinline__ int row_of(int j) const {
    return wr * (kFragR * 16) + j * 16 + (lane & 15);
  }
  __device__ __forceinline__ int col_of(int i) const {
    return wc * (kFragC * 16) + i * 16 + (lane >> 4) * 4;
  }
};

__device__ __forceinline__ uint32_t gemm_all(const GemmArgs &a) {
  return (uint32_t)a.tiles_c * ((uint32_t)a.main_r + (uint32_t)a.tail_r * (uint32_t)a.splits);
}

// A workgroup goes through tiles first, first + gridDim.x, ...: the next one's
// first steps are loaded while this one's sums are put away.
//   take(tile) is called before those loads, with the sums: what it loads is
//   there first; put(tile) after, and says whether the next tile may count
//   STORES memory operations behind them.
template <int STORES, class Tile, class Op, class Start, class Take, class Put>
__device__ __forceinline__ void gemm_tiles(Tile &t, const GemmArgs &a, Op, uint32_t first,
                                           const Start &start, const Take &take, const Put &put) {
  const uint32_t all = gemm_all(a);
  uint32_t id = first;
  if (id >= all) return;
  bool counted = false;
  t.at = gemm_place<Op, Tile::kC, Tile::kR>(a, id);
  t.prefetch(t.at);
  for (;;) {
    start();
    t.template run<STORES>(counted);
    t.fresh();
    take();
    id += gridDim.x;
    const bool more = id < all;
    GemmPlace next{};
    if (more) {
      next = gemm_place<Op, Tile::kC, Tile::kR>(a, id);
      t.prefetch(next);
    }
    t.fresh();
    counted = put();
    if (!more) break;
    t.at = next;
  }
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of 256 x 256 (one workgroup a CU) or 128 x 128 (two), and how many of
// their rows are summed whole and the others in how many parts of k, by what
// each would take on 256 CUs: rounds of workgroups, each its steps and what
// comes before and after them, and the parts' sums written and read. Measured
// in us: a step of a large tile 1.7, of a small one 1.2 (two at a time);
// before and after 8 and 6. Whole rounds come first, so that only what would
// leave most of the card idle at the end is split.
// Cross entropy with both gradients, by these rules, small tiles, large tiles,
// and without parts (us): 256 x 256 x 128 float32 43.5, 44.0, 66.7, 44.9;
// 400 x 5000 x 512 bf16 50, 50, 68, 83; 2000 x 8192 x 768 138, 143, 158, 155;
// 1000 x 30,522 x 384 float32 390, 402, 391, 1253; 4095 x 30,522 x 768 701, 776,
// 692, 896; 8192 x 100,000 x 1024 5206, 6612, 5147, 6666. Over 24 other sizes (64 to
// 8192 queries, 600 to 130,000 items, 76 to 1012 dims, every type) at most 5 % above
// the better of small and large tiles, the losses alone at most 6 %.
constexpr int kCus = 256;
struct TilePlan {
  bool big;
  int32_t tiles_c, main_r, tail_r, splits;
  double us;
  int64_t size() const { return big ? 256 : 128; }
  int64_t tail_row() const { return main_r * size(); }  // the first row of the tail
  int64_t all() const { return (int64_t)tiles_c * (main_r + (int64_t)tail_r * splits); }
  int64_t at_once() const { return big ? kCus : 2 * kCus; }
  uint32_t grid() const { return (uint32_t)(all() < at_once() ? all() : at_once()); }
  void give(GemmArgs *a) const {
    a->tiles_c = tiles_c;
    a->main_r = main_r;
    a->tail_r = tail_r;
    a->splits = splits;
  }
};
inline TilePlan plan_tiles(bool big, int64_t rows, int64_t cols, int64_t steps, int most_splits) {
  TilePlan best{};
  best.us = 1e300;
  const int64_t t = big ? 256 : 128, slots = big ? kCus : 2 * kCus;
  const int64_t tr = ceil_div(rows, t), tc = ceil_div(cols, t);
  const double step = big ? 1.7 : 1.2, around = big ? 8.0 : 6.0;
  const double whole = (double)steps * step + around;
  const auto offer = [&](int64_t main_r, int z, double us) {
    if (us < best.us) best = {big, (int32_t)tc, (int32_t)main_r, (int32_t)(tr - main_r), z, us};
  };
  offer(tr, 1, (double)ceil_div(tr * tc, slots) * whole);
  const int64_t rounds = tr * tc / slots, main_r = rounds * slots / tc;
  const int64_t tail = (tr - main_r) * tc;
  if (tail == 0) return best;
  const double values = (double)(rows - main_r * t) * (double)cols;
  // 2, 3, 4, 5, 6, 7, 8, 10, 12, ...: an eighth apart at the least
  for (int z = 2; z <= most_splits && z * 4 <= steps; z += z < 8 ? 1 : z / 8 * 2)
    offer(main_r, z,
          (double)rounds * whole +
              (double)ceil_div(tail * z, slots) * ((double)ceil_div(steps, z) * step + around) + 5.0 +
              (double)z * values * 8.0 / 4e6);
  return best;
}
inline TilePlan plan_tiles(int64_t rows, int64_t cols, int64_t steps, int most_splits) {
  const TilePlan small = plan_tiles(false, rows, cols, steps, most_splits);
  const TilePlan large = plan_tiles(true, rows, cols, steps, most_splits);
  return large.us < small.us ? large : small;
}

}  // namespace sps
