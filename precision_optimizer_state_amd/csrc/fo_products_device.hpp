// fo_products_device.hpp -- the matrix product that the products' kernels share:
//   out[c][r] = sum over k of C[c][k] * R[r][k]
// on the matrix cores.  Either operand may lie in memory by rows (rows r, k contiguous)
// or by columns (rows k, r contiguous).  What becomes of a tile of sums is the
// epilogue's (fo_products_kernels.hpp).
//
// A workgroup of WR x WC waves owns a tile of WR*FR*32 rows of R by WC*FC*32 rows of C
// and walks along k in steps of 128 bytes (64 elements of a 16-bit type, 32 floats).
// (Small tiles have two such groups of waves, which share each step's four sub-steps.)
// Operands go from memory straight into LDS, 16 bytes ("a piece") per lane, in a ring
// of NS stages.
//
// A wave multiplies FR fragments of 32 rows by FC of 32 rows.  A fragment is 16 bytes
// per lane: row lane % 32, elements of k from piece 2 s + lane / 32 of sub-step s.  One
// 16-bit matrix instruction takes a whole fragment (32x32x16); four float ones
// (32x32x2) take a float each: the order along k is permuted, the same way on both
// sides.  Sums are float32.  Lane l holds 16 sums of column c = l % 32 of the fragment
// pair, of rows r = 8 (i / 4) + 4 (l / 32) + i % 4: four neighbours in r at a time,
// which is the direction in which outputs are contiguous.
//
// LDS by rows: piece p of row r at place p ^ (r / 2 % 8) of the row's 128 bytes; the 16
// rows whose piece p is read together lie in the 16 different 16-byte columns of the 64
// banks.  (With r % 8 for r / 2 % 8 rows r and r + 8 share a column, and half of the
// reads' cycles were bank conflicts.)
// LDS by columns: a row of k holds the tile's pieces, permuted in fours by k so that
// the four rows of k that a transposing read touches (16-bit types: ds_read_b64_tr_b16,
// 16 lanes reading 4 rows of 16 elements get a column of 4 each) lie in different
// banks.  Floats are read one by one.
//
// What bounds it.  A step of a 256 x 256 tile of 16-bit elements is 256 matrix
// instructions of 32 cycles on 4 units, 0.85 us at 2.4 GHz; 8192 x 4096 x 128256 takes
// 1.67 us per step and round, 1318 TFLOP/s of 2500 (libraries' products of such sizes
// reach 1240 to 1430 on the same card).  The matrix units are busy 75 % of the cycles
// there and the clock has come down to 1.67 GHz: power is what is left to save.  With
// both operands a single row, all from L2, it reaches 1850.  Why so:
//   256 x 256 over 8 waves of 128 x 64: 0.75 fragment reads per matrix instruction, one
//   workgroup per compute unit.  Four waves of 128 x 128 read 0.5 and spill (1235
//   against 1300); waves 4 x 2 instead of 2 x 4 are 1 to 2 % slower; 128 x 128 tiles
//   reach 945 to 1065 where there are enough tiles for either.
//   The order of instructions in the main loop: 1274 before, 1300 with it, and 975 to
//   1110 for products of 768 columns.  Wave priorities change nothing.
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

// How a product's operands lie.
enum Form {
  ROWS_ROWS,      // both by rows
  DUAL_ROWS,      // both by rows; fragments of 32 rows of R alternate between r and r2
  COLS_ROWS,      // R by columns; with r2, steps of k from `joint` on are r2's
  COLS_COLS,      // both by columns
};

// One product: R is nr x k, C is nc x k.  `ld`: bytes from one row (of memory) to the
// next.  Everything is 16-byte aligned.  By rows k is a multiple of a step (padded with
// zeros).  By columns rows of memory are whole pieces long; C has a row for every k of
// its steps, of R there may be fewer (`k`, of each of r and r2): the last is read again
// for those, which C has as 0.
struct Product {
  const void* r;
  const void* r2;
  const void* c;
  int64_t r_ld, c_ld;
  int nr, nc;               // rows
  int k;                    // R by columns: rows of k
  int joint;                // COLS_ROWS: steps of r
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

// KS: groups of waves that share a tile's sub-steps (each has its own sums of every
// place of the tile, which are added at the end).
template <int WR, int WC, int FR, int FC, int NS, int KS>
struct Tile {
  static constexpr int R = WR * FR * 32, C = WC * FC * 32, group = WR * WC, groups = KS, waves = group * KS, threads = waves * 64;
  static constexpr int stage_bytes = (R + C) * kStepBytes, lds_bytes = stage_bytes * NS;
  static constexpr int loads = (R + C) / 8 / waves;            // of a wave, per stage
  static_assert((R + C) / 8 % waves == 0 && R / 8 % waves == 0, "loads are shared evenly");
};

// One operand's loads and reads.  N: rows of the tile; F: fragments of a wave.
// By rows.  DUAL: fragments of 32 rows alternate between two matrices.
template <typename T, int N, int F, int WAVES, bool DUAL>
struct ByRows {
  static constexpr int loads = N / 8 / WAVES;
  uint32_t off[loads], at[4];
  v4u buf[DUAL ? 2 : 1];

  // rows past the last are read as the last again (their sums are not used)
  // `sub`: the sub-step that this wave calls its first
  __device__ __forceinline__ void init(const void* base, const void* base2, int64_t ld, int row0, int rows, int k_bytes,
                                       int first, int sub, int lane, int wave) {
    const int mine = DUAL ? N / 2 : N;
#pragma unroll
    for (int i = 0; i < loads; ++i) {
      const int chunk = i * WAVES + wave, row = chunk * 8 + (lane >> 3), src = DUAL ? row / 64 * 32 + row % 32 : row;
      // (a load's rows begin at a multiple of 8, so r / 2 % 8 is 4 on its odd chunks and lane / 16)
      const uint32_t piece = (uint32_t)((lane & 7) ^ ((chunk & 1) * 4 + (lane >> 4))) * 16;
      off[i] = (uint32_t)min(src, rows - 1 - row0) * (uint32_t)ld + piece;
    }
    const uint32_t bytes = (uint32_t)(min(mine, rows - row0) - 1) * (uint32_t)ld + (uint32_t)k_bytes;
    buf[0] = buffer_of((const uint8_t*)base + (int64_t)row0 * ld, bytes);
    if constexpr (DUAL) buf[1] = buffer_of((const uint8_t*)base2 + (int64_t)row0 * ld, bytes);
#pragma unroll
    for (int s = 0; s < 4; ++s)
      at[s] = (uint32_t)(first * 32 + (lane & 31)) * kStepBytes + (uint32_t)(((2 * ((s + sub) & 3) + (lane >> 5)) ^ (lane >> 1 & 7)) * 16);
  }
  // load i of a step
  struct Step { uint32_t k; };
  __device__ __forceinline__ Step at_step(int step) const { return {(uint32_t)step * kStepBytes}; }
  __device__ __forceinline__ void fetch(const Step& step, int i, uint32_t lds, int wave) const {
    const int chunk = i * WAVES + wave;
    v4u b = buf[0];
    if constexpr (DUAL) {             // 4 loads of 8 rows make a fragment
#pragma unroll
      for (int e = 0; e < 4; ++e)
        b[e] = (uint32_t)__builtin_amdgcn_readfirstlane((int)(chunk / 4 & 1 ? buf[1][e] : buf[0][e]));
    }
    load_to_lds(b, off[i], step.k, lds + (uint32_t)chunk * 1024);
  }
  __device__ __forceinline__ v4u read(const uint8_t* lds, int s, int f) const {
    return *(const v4u*)(lds + at[s] + f * 32 * kStepBytes);
  }
};

// By columns.
template <typename T, int N, int F, int WAVES>
struct ByColumns {
  static constexpr int loads = N / 8 / WAVES, per = 16 / elem_bytes<T>, pieces = N / per, row_bytes = N * elem_bytes<T>;
  uint32_t off[loads], at[F];
  const uint8_t *base, *base2;
  int64_t ld;
  int k, joint, lane, left;

  // the place of piece p in row k of LDS
  static __device__ __forceinline__ int place(int k, int p) {
    if (is_f32<T>) return pieces >= 16 ? p ^ (k >> 2 & 1) << 3 : p;
    return pieces >= 16 ? p ^ (k & 3) << 2 : pieces == 8 ? p ^ (k >> 1 & 1) << 2 : p;
  }
  __device__ __forceinline__ void init(const void* b, const void* b2, int64_t ld_, int row0, int rows, int k_, int joint_,
                                       int first, int sub, int lane_, int wave) {
    base = (const uint8_t*)b + (int64_t)row0 * elem_bytes<T>;
    base2 = b2 ? (const uint8_t*)b2 + (int64_t)row0 * elem_bytes<T> : nullptr;
    ld = ld_; k = k_; joint = joint_; lane = lane_;
    left = (rows - row0 + per - 1) / per;           // pieces of a row from here on
#pragma unroll
    for (int i = 0; i < loads; ++i) off[i] = offset(i, wave, kStep<T>);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      if constexpr (is_f32<T>) {
        const int row = (first + f) * 32 + (lane & 31), kk = (lane >> 5) * 4;
        at[f] = (uint32_t)((sub * 8 + kk) * row_bytes + place(kk, row / 4) * 16 + row % 4 * 4);
      } else {
        const int i = lane & 15, kk = (lane >> 5) * 8 + i / 4, row = (first + f) * 32 + (lane >> 4 & 1) * 16 + i % 4 * 4;
        at[f] = (uint32_t)((sub * 16 + kk) * row_bytes + place(kk, row / 8) * 16 + row % 8 * 2);
      }
    }
  }
  // of load i from the step's first row of k, of which `rows` are there
  __device__ __forceinline__ uint32_t offset(int i, int wave, int rows) const {
    const int slot = (i * WAVES + wave) * 64 + lane, kk = slot / pieces, p = place(kk, slot % pieces);
    return (uint32_t)min(kk, rows - 1) * (uint32_t)ld + (uint32_t)min(p, left - 1) * 16;
  }
  struct Step { v4u buf; int rows; };
  __device__ __forceinline__ Step at_step(int step) const {
    const bool second = base2 && step >= joint;
    const int k0 = min((second ? step - joint : step) * kStep<T>, k - 1), rows = k - k0;
    return {buffer_of((second ? base2 : base) + (int64_t)k0 * ld,
                      (uint32_t)(min(rows, kStep<T>) - 1) * (uint32_t)ld + (uint32_t)left * 16), rows};
  }
  __device__ __forceinline__ void fetch(const Step& step, int i, uint32_t lds, int wave) const {
    const uint32_t o = step.rows < kStep<T> ? offset(i, wave, step.rows) : off[i];
    load_to_lds(step.buf, o, 0, lds + (uint32_t)(i * WAVES + wave) * 1024);
  }
  __device__ __forceinline__ v4u read(const uint8_t* lds, int s, int f) const {
    const uint8_t* p = lds + at[f];
    if constexpr (is_f32<T>) {
      v4u v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *(const uint32_t*)(p + (s * 8 + i) * row_bytes);
      return v;
    } else {
      typedef short s4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s4 lds_s4;
      const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + s * 16 * row_bytes));
      const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + (s * 16 + 4) * row_bytes));
      const v2u a = __builtin_bit_cast(v2u, lo), b = __builtin_bit_cast(v2u, hi);
      return (v4u){a[0], a[1], b[0], b[1]};
    }
  }
};

template <bool C, typename A, typename B> struct Pick { typedef A type; };
template <typename A, typename B> struct Pick<false, A, B> { typedef B type; };

// The sums of this wave: acc[i][j] of fragment i of R and j of C.
template <typename T, typename TL, int WR, int WC, int FR, int FC, int NS, Form FORM>
__device__ __forceinline__ void multiply(const Product& p, const Place& place, uint8_t* lds_raw, v16f (&acc)[FR][FC]) {
  constexpr bool dual = FORM == DUAL_ROWS, r_rows = FORM == ROWS_ROWS || dual, c_rows = FORM != COLS_COLS;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wr = wave % WR, wc = wave % TL::group / WR;
  constexpr int SUBS = 4 / TL::groups;                          // of a wave
  const int sub = wave / TL::group * SUBS;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds_raw;
  const int first = (int)((int64_t)place.slice * p.steps / p.slices);
  const int n = (int)((int64_t)(place.slice + 1) * p.steps / p.slices) - first;

  typename Pick<r_rows, ByRows<T, TL::R, FR, TL::waves, dual>, ByColumns<T, TL::R, FR, TL::waves>>::type R;
  typename Pick<c_rows, ByRows<T, TL::C, FC, TL::waves, false>, ByColumns<T, TL::C, FC, TL::waves>>::type C;
  if constexpr (r_rows) R.init(p.r, p.r2, p.r_ld, place.r * (dual ? TL::R / 2 : TL::R), p.nr, p.steps * kStepBytes, wr * FR, sub, lane, wave);
  else R.init(p.r, p.r2, p.r_ld, place.r * TL::R, p.nr, p.k, p.joint, wr * FR, sub, lane, wave);
  if constexpr (c_rows) C.init(p.c, nullptr, p.c_ld, place.c * TL::C, p.nc, p.steps * kStepBytes, wc * FC, sub, lane, wave);
  else C.init(p.c, nullptr, p.c_ld, place.c * TL::C, p.nc, p.steps * kStep<T>, 0, wc * FC, sub, lane, wave);

#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < FC; ++j) acc[i][j] = (v16f)(0.0f);

  // The sub-steps' work is interleaved by hand: each matrix instruction is followed by one
  // read of the next sub-step's fragments, and in a step's last sub-step by its share of
  // the loads of stage k + NS, so that neither a burst of reads nor one of loads leaves
  // the matrix unit idle.  The scheduling barriers keep that order.
  v4u fr[2][FR], fc[2][FC];
  constexpr int M = FR * FC, READS = FR + FC, RL = decltype(R)::loads, LOADS = TL::loads;
  auto read_one = [&](int n, int s, const uint8_t* buf) {       // R's first, C's, the rest of R's
    if (n == 0) fr[s & 1][0] = R.read(buf, s, 0);
    else if (n <= FC) fc[s & 1][n - 1] = C.read(buf + TL::R * kStepBytes, s, n - 1);
    else fr[s & 1][n - FC] = R.read(buf, s, n - FC);
  };
  // sub-step s; reads sub-step s + 1 (or the first) from `next`; then(m): after matrix instruction m
  auto sub_step = [&](int s, const uint8_t* next, auto&& then) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      acc[m / FC][m % FC] = mma<T>(fr[s & 1][m / FC], fc[s & 1][m % FC], acc[m / FC][m % FC]);
      if (m < READS) read_one(m, (s + 1) % SUBS, next);
      if (m == M - 1) {
#pragma unroll
        for (int n = M; n < READS; ++n) read_one(n, (s + 1) % SUBS, next);
      }
      then(m);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // loads [lo, hi) of a stage
  auto fetch = [&](const auto& r, const auto& c, int stage, int lo, int hi) {
    const uint32_t base = lds0 + (uint32_t)stage * TL::stage_bytes;
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      if (i >= lo && i < hi) {
        if (i < RL) R.fetch(r, i, base, wave);
        else C.fetch(c, i - RL, base + TL::R * kStepBytes, wave);
      }
  };

#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (s < n) fetch(R.at_step(first + s), C.at_step(first + s), s, 0, LOADS);
  if (n >= NS) wait_loads<(NS - 1) * TL::loads>();
  else wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < READS; ++i) read_one(i, 0, lds_raw);
  int stage = 0;
  auto step = [&](int k) {
    const int next = stage == NS - 1 ? 0 : stage + 1;
#pragma unroll
    for (int s = 0; s < SUBS - 1; ++s) sub_step(s, lds_raw + stage * TL::stage_bytes, [](int) {});
    // this wave has read all of stage k, and its loads of stage k + 1 have arrived when at
    // most those of later stages are under way
    if (NS > 2 && k + NS <= n) wait_loads<(NS - 2) * TL::loads>();
    else wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // ... and so have the others: stage k's place takes stage k + NS.  (The last step
    // reads what nothing uses: with matrix instructions on two paths their registers
    // would be copied from one to the other, and do not fit.)
    const bool more = k + NS < n;
    const auto r = R.at_step(first + min(k + NS, n - 1));
    const auto c = C.at_step(first + min(k + NS, n - 1));
    sub_step(SUBS - 1, lds_raw + next * TL::stage_bytes, [&](int m) {
      if (more) fetch(r, c, stage, m * LOADS / M, (m + 1) * LOADS / M);
    });
    stage = next;
  };
  // Float32 sums of long k: what 16 steps (512 terms) give is added to sums of its own,
  // where registers allow it (wide tiles' do not).  One token of 4096 columns is off by
  // 0.9e-6 of its norm instead of 1.7e-6, as much as a library's split product.
  if constexpr (is_f32<T> && FR * FC <= 4) {
    v16f sum[FR][FC];
#pragma unroll
    for (int i = 0; i < FR * FC; ++i) sum[i / FC][i % FC] = (v16f)(0.0f);
    for (int k = 0; k < n;) {
      for (const int stop = min(n, k + 16); k < stop; ++k) step(k);
#pragma unroll
      for (int i = 0; i < FR * FC; ++i) {
        sum[i / FC][i % FC] += acc[i / FC][i % FC];
        acc[i / FC][i % FC] = (v16f)(0.0f);
      }
    }
#pragma unroll
    for (int i = 0; i < FR * FC; ++i) acc[i / FC][i % FC] = sum[i / FC][i % FC];
  } else {
    for (int k = 0; k < n; ++k) step(k);
  }
  if constexpr (TL::groups == 2) {
    static_assert(TL::group * FR * FC * 4096 <= TL::lds_bytes, "sums of a group");
    uint8_t* mine = lds_raw + ((wave % TL::group) * FR * FC * 4 * 64 + lane) * 16;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < FR * FC * 4; ++n) {
      const v16f& a = acc[n / 4 / FC][n / 4 % FC];
      if (sub) *(v4f*)(mine + n * 1024) = (v4f){a[n % 4 * 4], a[n % 4 * 4 + 1], a[n % 4 * 4 + 2], a[n % 4 * 4 + 3]};
    }
    __syncthreads();
    if (!sub) {
#pragma unroll
      for (int n = 0; n < FR * FC * 4; ++n) {
        const v4f b = *(const v4f*)(mine + n * 1024);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n / 4 / FC][n / 4 % FC][n % 4 * 4 + e] += b[e];
      }
    }
  }
}

}  // namespace prod
}  // namespace fo
