// fo_products_device.hpp -- the matrix product that the products' kernels share:
//   out[c][r] = sum over k of C[c][k] * R[r][k]
// for two operands whose rows are contiguous along k, on the matrix cores.
// What becomes of a tile of sums is the epilogue's (fo_products_kernels.hpp).
//
// A workgroup of WR x WC waves owns a tile of WR*FR*32 rows of R by WC*FC*32 rows
// of C and walks along k in steps of 128 bytes (64 elements of a 16-bit type, 32
// floats).  Rows go from memory straight into LDS, 16 bytes per lane, in a ring of
// NS stages.  Piece c (16 bytes) of row r goes to place c ^ (r / 2 % 8) of the row's
// 128 bytes: the 16 rows whose piece c is read together then lie in the 16 different
// 16-byte columns of the 64 banks.  (With r % 8 for r / 2 % 8 rows r and r + 8 share
// a column, and half of the reads' cycles were bank conflicts.)
//
// A wave multiplies FR fragments of 32 rows by FC of 32 rows.  A fragment is 16
// bytes per lane: row lane % 32, piece 2 s + lane / 32 of sub-step s.  One 16-bit
// matrix instruction takes a whole fragment (32x32x16); four float ones (32x32x2)
// take a float each: the order along k is permuted, the same way on both sides.
// Sums are float32.  Lane l holds 16 sums of column c = l % 32 of the fragment
// pair, of rows r = 8 (i / 4) + 4 (l / 32) + i % 4: four neighbours in r at a time,
// which is the direction in which outputs are contiguous.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fo_rows_device.hpp"

namespace fo {
namespace prod {

using rows::Bf16;
using rows::Fp16;
using rows::F32;
using rows::is_f32;

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kStepBytes = 128;                 // of k per step
template <typename T> constexpr int elem_bytes = is_f32<T> ? 4 : 2;
template <typename T> constexpr int kStep = kStepBytes / elem_bytes<T>;

template <typename T>
__device__ __forceinline__ v16f mma(v4u r, v4u c, v16f acc) {
  if constexpr (is_f32<T>) {
    const v4f fr = __builtin_bit_cast(v4f, r), fc = __builtin_bit_cast(v4f, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(fr[i], fc[i], acc, 0, 0, 0);
    return acc;
  } else if constexpr (__is_same(T, Bf16)) {
    typedef __bf16 b8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, r), __builtin_bit_cast(b8, c), acc, 0, 0, 0);
  } else {
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, r), __builtin_bit_cast(h8, c), acc, 0, 0, 0);
  }
}

// One product: R is nr x k, C is nc x k, rows `ld` bytes apart, k a multiple of a
// step (operands are padded with zeros), everything 16-byte aligned.  With two
// matrices in R (`r2`) fragments of 32 rows alternate between them.
struct Product {
  const void* r;
  const void* r2;
  const void* c;
  int64_t r_ld, c_ld;       // bytes
  int nr, nc;               // rows
  int steps;                // of k
  int tiles_r, tiles_c;
  int slices;               // of k: slice s takes steps [s * steps / slices, (s + 1) * steps / slices)
};

// Which tile and slice a workgroup takes.  Workgroups go to the 8 XCDs in turn, each
// with an L2 of its own: an XCD gets consecutive tiles, ordered so that those that
// run together share rows of both operands (8 tiles of C by as many of R as fit).
struct Place { int r, c, slice; };

__device__ __forceinline__ Place place(const Product& p) {
  const int total = p.tiles_r * p.tiles_c * p.slices, id = blockIdx.x;
  const int xcd = id & 7, q = total >> 3, rem = total & 7;
  int t = xcd * q + min(xcd, rem) + (id >> 3);
  const int per_slice = p.tiles_r * p.tiles_c, slice = t / per_slice;
  t -= slice * per_slice;
  const int band = 8 * p.tiles_r, first = t / band * 8, width = min(8, p.tiles_c - first);
  t -= first * p.tiles_r;
  return {t / width, first + t % width, slice};
}

// 64 lanes x 16 bytes from memory into 1 KiB of LDS at `lds` (the same for the whole
// wave).  Written as assembly because the compiler, told of a load into LDS, waits
// for it before the next read of any other part of LDS; the waits are in the kernel.
// (M0 is a reserved register, which nothing else in these kernels uses.)
__device__ __forceinline__ void load_to_lds(v4u rsrc, uint32_t lane_offset, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :: "v"(lane_offset), "s"(rsrc), "s"(offset), "s"(lds) : "memory");
}

__device__ __forceinline__ v4u buffer_of(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return (v4u){(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

template <int N> __device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(N) : "memory");
}

template <int WR, int WC, int FR, int FC, int NS>
struct Tile {
  static constexpr int R = WR * FR * 32, C = WC * FC * 32, waves = WR * WC, threads = waves * 64;
  static constexpr int stage_bytes = (R + C) * kStepBytes, lds_bytes = stage_bytes * NS;
  static constexpr int loads = (R + C) / 8 / waves;            // of a wave, per stage
  static_assert((R + C) / 8 % waves == 0 && R / 8 % waves == 0, "loads are shared evenly");
};

// The sums of this wave: acc[i][j] of fragment i of R and j of C.
template <typename T, typename TL, int WR, int WC, int FR, int FC, int NS, bool DUAL>
__device__ __forceinline__ void multiply(const Product& p, const Place& at, uint8_t* lds_raw, v16f (&acc)[FR][FC]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds_raw;
  const int r0 = at.r * (DUAL ? TL::R / 2 : TL::R), c0 = at.c * TL::C;
  const int first = (int)((int64_t)at.slice * p.steps / p.slices);
  const int n = (int)((int64_t)(at.slice + 1) * p.steps / p.slices) - first;

  // offsets of this lane's loads from the tile's first row; rows past the last are
  // read as the last one again (their sums are not used)
  constexpr int LR = TL::R / 8 / TL::waves, LC = TL::C / 8 / TL::waves;
  uint32_t off[LR + LC];
  v4u rs[DUAL ? 2 : 1], cs;
  // (a load's rows begin at a multiple of 8, so r / 2 % 8 is 4 on its odd chunks and lane / 16)
  auto piece = [&](int i) { return (uint32_t)((lane & 7) ^ (((i * TL::waves + wave) & 1) * 4 + (lane >> 4))) * 16; };
#pragma unroll
  for (int i = 0; i < LR; ++i) {
    const int row = (i * TL::waves + wave) * 8 + (lane >> 3);
    const int src = DUAL ? row / 64 * 32 + row % 32 : row;
    off[i] = (uint32_t)min(src, p.nr - 1 - r0) * (uint32_t)p.r_ld + piece(i);
  }
#pragma unroll
  for (int i = 0; i < LC; ++i) {
    const int row = (i * TL::waves + wave) * 8 + (lane >> 3);
    off[LR + i] = (uint32_t)min(row, p.nc - 1 - c0) * (uint32_t)p.c_ld + piece(i);
  }
  const uint32_t k_bytes = (uint32_t)p.steps * kStepBytes;
  const uint32_t r_rows = (uint32_t)min(DUAL ? TL::R / 2 : TL::R, p.nr - r0), c_rows = (uint32_t)min(TL::C, p.nc - c0);
  rs[0] = buffer_of((const uint8_t*)p.r + (int64_t)r0 * p.r_ld, (r_rows - 1) * (uint32_t)p.r_ld + k_bytes);
  if constexpr (DUAL) rs[1] = buffer_of((const uint8_t*)p.r2 + (int64_t)r0 * p.r_ld, (r_rows - 1) * (uint32_t)p.r_ld + k_bytes);
  cs = buffer_of((const uint8_t*)p.c + (int64_t)c0 * p.c_ld, (c_rows - 1) * (uint32_t)p.c_ld + k_bytes);

  auto fetch = [&](int step, int stage) {
    const uint32_t k = (uint32_t)(first + step) * kStepBytes;
    const uint32_t base = lds0 + (uint32_t)stage * TL::stage_bytes;
#pragma unroll
    for (int i = 0; i < LR; ++i) {
      const int chunk = i * TL::waves + wave;
      if constexpr (DUAL) {
        // 4 loads of 8 rows make a fragment; waves are a multiple of 4 or a load's
        // fragment is its wave's to find
        v4u b;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
          b[k4] = (uint32_t)__builtin_amdgcn_readfirstlane((int)(chunk / 4 & 1 ? rs[1][k4] : rs[0][k4]));
        load_to_lds(b, off[i], k, base + (uint32_t)chunk * 1024);
      } else {
        load_to_lds(rs[0], off[i], k, base + (uint32_t)chunk * 1024);
      }
    }
#pragma unroll
    for (int i = 0; i < LC; ++i)
      load_to_lds(cs, off[LR + i], k, base + TL::R * kStepBytes + (uint32_t)(i * TL::waves + wave) * 1024);
  };

#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FC; ++j) acc[i][j] = (v16f)(0.0f);

  const int wr = wave % WR, wc = wave / WR;
  uint32_t at_r[4], at_c[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t x = (uint32_t)(lane & 31) * kStepBytes + (uint32_t)(((2 * s + (lane >> 5)) ^ (lane >> 1 & 7)) * 16);
    at_r[s] = x + (uint32_t)(wr * FR * 32) * kStepBytes;
    at_c[s] = x + (uint32_t)(TL::R + wc * FC * 32) * kStepBytes;
  }

  // Fragments are read one sub-step ahead of the matrix instructions that use them, and
  // the first of a step before the last instructions of the step before: no wave waits
  // for LDS with its matrix unit idle.  The scheduling barriers keep that order.
  v4u fr[2][FR], fc[2][FC];
  auto read = [&](int s, int stage) {
    const uint8_t* buf = lds_raw + stage * TL::stage_bytes;
#pragma unroll
    for (int i = 0; i < FR; ++i) fr[s & 1][i] = *(const v4u*)(buf + at_r[s] + i * 32 * kStepBytes);
#pragma unroll
    for (int j = 0; j < FC; ++j) fc[s & 1][j] = *(const v4u*)(buf + at_c[s] + j * 32 * kStepBytes);
  };
  auto use = [&](int s) {
#pragma unroll
    for (int i = 0; i < FR; ++i)
#pragma unroll
      for (int j = 0; j < FC; ++j) acc[i][j] = mma<T>(fr[s & 1][i], fc[s & 1][j], acc[i][j]);
  };

#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (s < n) fetch(s, s);
  if (n >= NS) wait_loads<(NS - 1) * TL::loads>();
  else wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  read(0, 0);
  int stage = 0;
  for (int k = 0; k < n; ++k) {
    const int next = stage == NS - 1 ? 0 : stage + 1;
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      read(s + 1, stage);
      __builtin_amdgcn_sched_barrier(0);
      use(s);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (k + 1 < n) {
      // this wave has read all of stage k, and its loads of stage k + 1 have arrived
      // when at most those of later stages are under way
      if (NS > 2 && k + NS <= n) wait_loads<(NS - 2) * TL::loads>();
      else wait_loads<0>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      // ... and so have the others: stage k's place takes stage k + NS
      read(0, next);
      __builtin_amdgcn_sched_barrier(0);
      if (k + NS < n) fetch(k + NS, stage);
    }
    use(3);
    stage = next;
  }
}

}  // namespace prod
}  // namespace fo
