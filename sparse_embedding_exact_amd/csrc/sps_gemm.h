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

// float32 as three planes of bf16
struct OpF32 : OpBf16 {
  using Type = float;
  static constexpr int kPlanes = 3;
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

// k_bytes of every row take part (a multiple of 16). With planes the six
// products of planes that reach 2^-24 of a product are summed one after
// another, as if k were six times as long. splits > 1: workgroup (tile, z)
// sums the z-th part of the steps.
struct GemmArgs {
  GemmOperand q, p;
  int64_t k_bytes;
  int64_t k_rows;  // of a turned q
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

// Four values of a type, side by side.
template <typename T>
struct alignas(4 * sizeof(T)) Quad {
  T e[4];
};
template <typename T>
__device__ __forceinline__ Quad<T> quad_of(const float v[4]) {
  return {{from_f32<T>(v[0]), from_f32<T>(v[1]), from_f32<T>(v[2]), from_f32<T>(v[3])}};
}

typedef __attribute__((address_space(3))) uint8_t lds_u8;

template <class Op, int TC, int TR, int WC, int WR, bool QT = false>
struct GemmTile {
  static constexpr int kThreads = 64 * WC * WR;
  static constexpr int kC = TC, kR = TR;
  static constexpr int kFragC = TC / WC / 16, kFragR = TR / WR / 16;
  static constexpr int kBuf = (TC + TR) * kStep;  // bytes of one step
  static constexpr int kLds = 2 * kBuf;
  static constexpr int kRowsLoad = 8 * WC * WR;   // rows that one load of every wave fills
  static constexpr int kLoadsP = TC / kRowsLoad, kLoadsQ = TR / kRowsLoad;
  static_assert(TC % kRowsLoad == 0 && TR % kRowsLoad == 0, "whole loads");
  static_assert(kLds <= 160 * 1024, "LDS");
  using Acc = typename Op::Acc;
  using Frag = typename Op::Frag;

  Acc acc[kFragC][kFragR];

  // This wave's loads and reads are done, and behind the barrier every wave's.
  static __device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kFragC; ++i)
#pragma unroll
      for (int j = 0; j < kFragR; ++j) acc[i][j] = Acc{};
  }
  // Sums that go on from those in rows of cols values.
  __device__ __forceinline__ void start(const float *before, int64_t rows, int64_t cols, int64_t row0,
                                        int64_t col0) {
#pragma unroll
    for (int j = 0; j < kFragR; ++j) {
      const int64_t r = row0 + row_of(j);
#pragma unroll
      for (int i = 0; i < kFragC; ++i) {
        const int64_t c = col0 + col_of(i);
        const float *const x = before + r * cols + c;
        if (r < rows && c + 4 <= cols) {
          const Four<float> f = *reinterpret_cast<const Four<float> *>(x);
          acc[i][j] = Acc{f.e[0], f.e[1], f.e[2], f.e[3]};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = r < rows && c + e < cols ? x[e] : 0.0f;
        }
      }
    }
  }

  // Adds the sum over steps [begin, end) for the tile at (row0, col0). The steps are
  // taken from the turn-th on, round: rows whose length is a large power of two
  // have equal steps in few of L2's channels, and neighbouring tiles would ask
  // for them at once.
  __device__ __forceinline__ void run(const GemmArgs &a, int64_t row0, int64_t col0, int begin,
                                      int end, uint8_t *lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wc = wave % WC, wr = wave / WC;
    if (begin >= end) return;

    const uint32_t ld_p = (uint32_t)a.p.ld, ld_q = (uint32_t)a.q.ld;
    const auto left = [](int64_t rows, int64_t first, int64_t ld, int64_t in = 0) {
      const int64_t b = (rows - first) * ld - in;  // rows past the last read as zeros
      return (int)(b < (int64_t)kMostBytes ? b : (int64_t)kMostBytes);
    };
    const int size_p = left(a.p.rows, col0, a.p.ld);
    const int size_q = QT ? 0 : left(a.q.rows, row0, a.q.ld);
    uint8_t *const base_p = const_cast<uint8_t *>(a.p.base) + col0 * a.p.ld;
    uint8_t *const base_q = const_cast<uint8_t *>(a.q.base) + (QT ? row0 * 2 : row0 * a.q.ld);

    // this lane's place in a load: row lane / 8 of the wave's eight, and the chunk that belongs there
    const uint32_t row = (uint32_t)(wave * 8 + (lane >> 3));
    const uint32_t chunk = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
    const uint32_t off_p = row * ld_p + chunk;
    // Turned: 1024 bytes are 1024 / (2 TR) rows of k. A transposing read takes 32 bytes of 16 of
    // them, rows k and k + 8 apart among them: pair p of 16-byte chunks of row k stands at p ^ turn(k),
    // turn(k) = k % 4 + 4 (k / 8 % 2), so that 8 rows meet every bank once.
    constexpr int kPlaces = TR * 2 / 16;
    const uint32_t k_row = (uint32_t)(wave * (64 / kPlaces) + lane / kPlaces), place_q = (uint32_t)(lane % kPlaces);
    const uint32_t turn = (k_row & 3) | (k_row >> 3 & 1) << 2;
    const uint32_t off_q = QT ? k_row * ld_q + (place_q ^ (turn << 1)) * 16 : row * ld_q + chunk;
    constexpr int kNextQ = QT ? (64 / kPlaces) * WC * WR : kRowsLoad;  // rows between a wave's loads
    static_assert(!QT || kNextQ % 16 == 0, "one turn(k) for all loads of a lane");

    const uint32_t k_end = (uint32_t)a.k_bytes;  // of one segment
    const int many = end - begin;
    int at_step = begin + (int)(((uint32_t)(col0 / TC) * 2u) % (uint32_t)many);
    int seg = 0;
    uint32_t k;
    const auto place = [&](int step) {
      if constexpr (Op::kPlanes > 1) {
        const int steps = (int)((k_end + kStep - 1) / kStep);
        seg = step / steps;
        k = (uint32_t)(step - seg * steps) * kStep;
      } else {
        k = (uint32_t)step * kStep;
      }
    };
    place(at_step);
    auto load = [&](uint8_t *buf) {
      uint8_t *const b = buf + wave * 1024;
      const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(
          base_p + (Op::kPlanes > 1 ? seg_p(seg) * a.p.plane : 0), 0, size_p, 0x00020000);
      const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
          base_q + (Op::kPlanes > 1 ? seg_q(seg) * a.q.plane : 0) +
              (QT ? (int64_t)(k / 2) * a.q.ld : 0),
          0, QT ? left(a.k_rows, (int64_t)(k / 2), a.q.ld, row0 * 2) : size_q, 0x00020000);
      // past the end of k: an offset past the buffer's, which reads zeros
      const bool in = k + chunk < k_end;
      const uint32_t at_p = in ? off_p + k : 0x80000000u;
      const uint32_t at_q = QT ? off_q : in ? off_q + k : 0x80000000u;
#pragma unroll
      for (int i = 0; i < kLoadsP; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (lds_u8 *)(b + i * kRowsLoad * kStep), 16,
                                                 (int)(at_p + (uint32_t)i * kRowsLoad * ld_p), 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kLoadsQ; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (lds_u8 *)(b + (TC + i * kRowsLoad) * kStep), 16,
                                                 (int)(at_q + (uint32_t)i * kNextQ * ld_q), 0, 0, 0);
      if (++at_step == end) {
        at_step = begin;
        place(begin);
      } else {
        k += kStep;
        if (Op::kPlanes > 1 && k >= k_end) {
          k = 0;
          ++seg;
        }
      }
    };

    // a fragment: row lane % 16, bytes 16 (lane / 16) of 64; the other 64 bytes are places ^ 4
    const int at0 = (lane & 15) * kStep + (((lane >> 4) ^ (lane & 7)) * 16), at1 = at0 ^ 64;
    const int from_p = wc * (kFragC * 16) * kStep, from_q = (TC + wr * (kFragR * 16)) * kStep;
    // turned: four lanes' 8 bytes are 16 columns of a row of k, 16 lanes' four rows, and a lane
    // receives a column of them: rows 8 (lane / 16) to + 3 of 32, and the four behind with a second read
    int turned[kFragR];
#pragma unroll
    for (int j = 0; j < kFragR; ++j) {
      const int four = (lane & 15) >> 2, k_at = (lane >> 4) * 8 + four;
      turned[j] = TC * kStep + k_at * TR * 2 +
                  ((wr * kFragR + j) ^ (four | ((lane >> 4) & 1) << 2)) * 32 + (lane & 3) * 8;
    }
    auto read_p = [&](const uint8_t *b, bool half, Frag (&p)[kFragC]) {
#pragma unroll
      for (int i = 0; i < kFragC; ++i)
        p[i] = *reinterpret_cast<const Frag *>(b + from_p + i * 16 * kStep + (half ? at1 : at0));
    };
    auto read_q = [&](const uint8_t *b, bool half, Frag (&q)[kFragR]) {
      if constexpr (QT) {
        // In assembly, since the compiler makes the builtin wait for every load to LDS on its way,
        // also those to the other buffer; the block ends with its own wait.
        static_assert(kFragR == 4, "four fragments a block");
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        s16x4 x[8];
        uint32_t at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          at[j] = (uint32_t)(uintptr_t)(lds_u8 *)const_cast<uint8_t *>(b) + turned[j] +
                  (half ? 32 * TR * 2 : 0);
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
            : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(4 * TR * 2)
            : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const s16x4 lo = x[2 * j], hi = x[2 * j + 1];
          const s16x8 both = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          q[j] = __builtin_bit_cast(Frag, both);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kFragR; ++j)
          q[j] = *reinterpret_cast<const Frag *>(b + from_q + j * 16 * kStep + (half ? at1 : at0));
      }
    };
    // Half a step from registers, while the next half is read into others.
    auto half_step = [&](Frag (&p)[kFragC], Frag (&q)[kFragR], bool more, const uint8_t *b, bool half,
                         Frag (&pn)[kFragC], Frag (&qn)[kFragR]) {
      if (more && !QT) read_q(b, half, qn);
      if (more) read_p(b, half, pn);
#pragma unroll
      for (int i = 0; i < kFragC; ++i) {
#pragma unroll
        for (int j = 0; j < kFragR; ++j) acc[i][j] = Op::mma(p[i], q[j], acc[i][j]);
        if (QT && i == kFragC / 2 - 1) {
          __builtin_amdgcn_sched_barrier(0);
          if (more) read_q(b, half, qn);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (!QT) {  // matrix instructions between the reads
        constexpr int kReads = kFragC + kFragR, kEach = kFragC * kFragR / kReads;
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };

    // Behind the barrier in a step's middle its buffer has been read to the end and is loaded again,
    // and the next step, which had a whole step's time, is in the other.
    Frag p0[kFragC], q0[kFragR], p1[kFragC], q1[kFragR];
    load(lds);
    arrive();
    if (many > 1) load(lds + kBuf);
    read_q(lds, false, q0);
    read_p(lds, false, p0);
    __builtin_amdgcn_sched_barrier(0);
    int here = 0;
    for (int s = 0; s < many; ++s) {
      half_step(p0, q0, true, lds + here, true, p1, q1);
      arrive();
      if (s + 2 < many) load(lds + here);
      __builtin_amdgcn_sched_barrier(0);
      here ^= kBuf;
      half_step(p1, q1, s + 1 < many, lds + here, false, p0, q0);
    }
    arrive();  // LDS is free for what follows
  }

  // Rows out of the registers' layout (16 rows of four values a lane) into whole runs: 16 rows at
  // a time go through this wave's own part of LDS, whose rows are 16 bytes longer than a run, so
  // that 16 lanes of 16 rows meet every bank once. Stores of 16-byte runs of 16 rows each reach
  // 3.2 TB/s, runs of 256 bytes and more what a fill does.
  static constexpr int kWaveLds = kLds / (WC * WR);
  template <typename T>
  static constexpr int kRun = TC / WC * (int)sizeof(T);
  template <typename T>
  struct __attribute__((packed, aligned(sizeof(T)))) Words {
    uint32_t w[4];
  };
  __device__ __forceinline__ uint8_t *wave_lds(uint8_t *lds) const {
    return lds + (threadIdx.x >> 6) * kWaveLds;
  }
  // This lane's four values of column group i, as 4 sizeof(T) bytes.
  template <typename T, typename W>
  __device__ __forceinline__ void stage(uint8_t *mine, int i, const W &v) const {
    static_assert(sizeof(W) == 4 * sizeof(T), "four values");
    static_assert(16 * (kRun<T> + 16) <= kWaveLds, "LDS");
    const int lane = threadIdx.x & 63;
    typedef uint32_t Bits __attribute__((ext_vector_type(sizeof(T))));
    *reinterpret_cast<Bits *>(mine + (lane & 15) * (kRun<T> + 16) +
                              (i * 16 + (lane >> 4) * 4) * (int)sizeof(T)) = __builtin_bit_cast(Bits, v);
  }
  // The staged 16 rows to `out` (row 0 of them, this wave's first column) for `rows` rows and
  // `cols` columns at the most.
  template <typename T>
  __device__ __forceinline__ void store(const uint8_t *mine, T *out, int64_t ld, int64_t rows,
                                        int64_t cols) const {
    constexpr int kLanes = kRun<T> / 16, kOnce = 64 / kLanes, V = 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 63;
    const int in = lane % kLanes;
    if (lane >= kOnce * kLanes) return;
#pragma unroll
    for (int r = 0; r < (16 + kOnce - 1) / kOnce; ++r) {
      const int row = r * kOnce + lane / kLanes;
      if (row >= 16 || row >= rows) continue;
      const u32x4 w = *reinterpret_cast<const u32x4 *>(mine + row * (kRun<T> + 16) + in * 16);
      T *const to = out + row * ld + in * V;
      if ((in + 1) * V <= cols) {
        *reinterpret_cast<Words<T> *>(to) = {{w[0], w[1], w[2], w[3]}};
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (in * V + e < cols) {
            const uint32_t u = w[e * (int)sizeof(T) / 4];
            if constexpr (sizeof(T) == 4) to[e] = __builtin_bit_cast(T, u);
            else to[e] = __builtin_bit_cast(T, (uint16_t)(u >> (16 * (e & 1))));
          }
      }
    }
  }
  // First row of row group j and first column of this wave in the tile.
  __device__ __forceinline__ int rows_at(int j) const {
    return ((threadIdx.x >> 6) / WC) * (kFragR * 16) + j * 16;
  }
  __device__ __forceinline__ int cols_at() const { return ((threadIdx.x >> 6) % WC) * (kFragC * 16); }

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
template <class Op, int TC, int TR>
__device__ __forceinline__ GemmPlace gemm_place(const GemmArgs &a) {
  GemmPlace g;
  int tc, tr;
  const uint32_t tiles = (uint32_t)a.tiles_c * (uint32_t)a.tiles_r;
  g.z = (int32_t)(blockIdx.x / tiles);
  tile_of(blockIdx.x % tiles, a.tiles_c, a.tiles_r, &tc, &tr);
  g.row0 = (int64_t)tr * TR;
  g.col0 = (int64_t)tc * TC;
  const int steps = (int)((a.k_bytes + kStep - 1) / kStep) * (Op::kPlanes > 1 ? kSegments : 1);
  g.begin = (int)((int64_t)steps * g.z / a.splits);
  g.end = (int)((int64_t)steps * (g.z + 1) / a.splits);
  return g;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of 256 x 256 (one workgroup a CU) or 128 x 128 (two), and into how
// many parts k goes, by what each would take on 256 CUs: rounds of workgroups,
// each its steps and what comes before and after them, and sums of parts
// written and read. Measured in us: a step of a large tile 1.7, of a small one
// 1.2 (two at a time); before and after 8 and 6.
struct TilePlan {
  bool big;
  int32_t splits;
};
inline TilePlan plan_tiles(int64_t rows, int64_t cols, int64_t steps, int most_splits) {
  TilePlan best{false, 1};
  double least = 1e300;
  for (int big = 0; big < 2; ++big) {
    const int64_t t = big ? 256 : 128, slots = big ? 256 : 512;
    const int64_t tiles = ceil_div(rows, t) * ceil_div(cols, t);
    for (int z = 1; z <= most_splits && (z == 1 || z * 4 <= steps); ++z) {
      const double each = (double)ceil_div(steps, z) * (big ? 1.7 : 1.2) + (big ? 8.0 : 6.0);
      const double join = z > 1 ? 5.0 + (double)z * (double)rows * (double)cols * 8.0 / 4e6 : 0.0;
      const double us = (double)ceil_div(tiles * z, slots) * each + join;
      if (us < least) {
        least = us;
        best = {big != 0, z};
      }
    }
  }
  return best;
}

}  // namespace sps
