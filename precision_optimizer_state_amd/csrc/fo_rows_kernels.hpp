// fo_rows_kernels.hpp -- HIP kernels (gfx950) of the row operators: dropout,
// layer norm / RMS norm and the fused dropout + residual sum + norm, forward
// and backward.
//
//   forward   h = residual + keep * x / (1 - p), rounded to the rows' type
//             (h = x without a residual);  m = mean(h), 0 for RMS;
//             r = 1 / sqrt(mean((h - m)^2) + eps);  y = (h - m) r w + b
//   backward  g = dy w;  u = (h - m) r;
//             d = r (g - mean(g) - u mean(g u)) + dh  (no mean(g) for RMS);
//             dx = keep * d / (1 - p);  dw = sum over rows of dy u;
//             db = sum over rows of dy
//
// All arithmetic is float32, means and sums included; each output is rounded
// once.  The statistics are those of h after its rounding, so that the backward
// pass, which reads h, is the gradient of what the forward pass returned.
#pragma once

#include "fo_rows_device.hpp"

namespace fo {
namespace rows {

constexpr int BLOCK = 256;

struct DropoutArgs {
  const void* x;
  void* y;
  int64_t rows, cols, x_ld;
  DropArgs drop;
};

struct FwdArgs {
  const void *x, *residual, *weight, *bias;
  void *h, *y;
  float *mean, *rstd;
  int64_t rows, first_row, x_ld, residual_ld;     // first_row: of this launch (k_norm_fwd)
  int cols, wdtype, rms, dropping;
  float eps;
  // Sums over a row are those of values times sum_scale = 4^-k and of squares of
  // values times square_scale = 2^-k, with 4^k the first power of 4 that reaches cols:
  // they overflow only where the mean itself would.  mean_scale = 4^k / cols makes
  // means of them.  Powers of two commute with every rounding of normal numbers.
  float sum_scale, square_scale, mean_scale;
  DropArgs drop;
};

struct BwdArgs {
  const void *dy, *dh, *h, *weight;
  const float *mean, *rstd;
  void *d, *dx;
  float* partial;              // [2][splits][cols]: dw, db
  int64_t rows, dy_ld, dh_ld, h_ld;
  int cols, wdtype, rms, splits;
  float inv_cols;
  DropArgs drop;
};

__device__ __forceinline__ int chunks_of(int cols) { return (cols + 7) >> 3; }

// ---------------------------------------------------------------------------
// dropout (the gradient is the same call on the output's gradient)
// ---------------------------------------------------------------------------
// HBM bound: 400000 x 1024 bf16 270 us, 6.1 TB/s (a copy of it without a mask runs
// at the same rate, see DropArgs); the generator hides behind the stream.  Chunks
// lie one after another in memory (FLAT: packed rows of whole chunks) or are found
// by one division (Index: in 32 bits where the number of chunks and a column allow
// it).  Two chunks per thread, loaded before either is worked on.
constexpr int DROP_PER = 2;

template <typename T, bool FLAT, typename Index>
__global__ __launch_bounds__(BLOCK) void k_dropout(DropoutArgs a) {
  typedef typename T::raw raw;
  const Index nch = (Index)((a.cols + 7) >> 3);
  const Index total = (Index)(a.rows * (int64_t)nch);
  const DropKey key = drop_key(a.drop);
  const int64_t step = (int64_t)gridDim.x * (BLOCK * DROP_PER);
  for (int64_t base = (int64_t)blockIdx.x * (BLOCK * DROP_PER) + threadIdx.x; base < (int64_t)total; base += step) {
    Chunk<T> in[DROP_PER];
    int64_t at[DROP_PER];
    int col[DROP_PER], end[DROP_PER], cnt[DROP_PER];
#pragma unroll
    for (int v = 0; v < DROP_PER; ++v) {
      const int64_t i = base + v * BLOCK;
      const bool live = i < (int64_t)total;
      if constexpr (FLAT) {
        at[v] = i * 8;
        cnt[v] = live ? 8 : 0;
        in[v] = load_part<T>((const raw*)a.x + at[v], 0, cnt[v]);
      } else {
        const Index r = live ? (Index)i / nch : 0, c = live ? ((Index)i - r * nch) * 8 : 0;
        // columns of 64 bits are counted from the chunk before, as far as the chunk after
        const int64_t from = sizeof(Index) == 8 && c > 8 ? (int64_t)c - 8 : 0, left = a.cols - from;
        end[v] = sizeof(Index) == 8 && left > 24 ? 24 : (int)left;
        col[v] = live ? (int)((int64_t)c - from) : end[v];
        at[v] = (int64_t)r * a.cols + (int64_t)c;
        cnt[v] = end[v] - col[v];
        in[v] = load_part<T>((const raw*)a.x + (int64_t)r * a.x_ld + from, col[v], end[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < DROP_PER; ++v) {
      if (cnt[v] <= 0) continue;
      if constexpr (!FLAT) settle_part<T>(in[v], col[v], end[v]);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = elem<T>(in[v], j);
      drop_chunk(a.drop, key, (uint64_t)(base + v * BLOCK), f);
      store_chunk<T>((raw*)a.y + at[v], to_chunk<T>(f), cnt[v]);
    }
  }
}

// ---------------------------------------------------------------------------
// norms
// ---------------------------------------------------------------------------
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 32; s; s >>= 1) v += __shfl_xor(v, s, 64);
  return v;
}

// sum over the workgroup, in every thread; `red` holds one float per wave
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  __syncthreads();                       // the previous sum has been read
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) s += red[i];
  return s;
}

// residual + dropout(x) of one chunk
template <typename T>
__device__ __forceinline__ Chunk<T> join(const Chunk<T>& x, const Chunk<T>& residual, bool dropping, const DropArgs& d,
                                         const DropKey& key, uint64_t index) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = elem<T>(x, j);
  if (dropping) drop_chunk(d, key, index, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] += elem<T>(residual, j);
  return to_chunk<T>(f);
}

// 1 / sqrt(v) to one unit in the last place: the hardware estimate where v is
// well inside the normal range (it takes subnormals for 0), else the IEEE form
__device__ __forceinline__ float rsqrt_of(float v) {
  return v > 0x1p-100f ? __builtin_amdgcn_rsqf(v) : 1.0f / sqrtf(v);
}

// ---------------------------------------------------------------------------
// sums over the lanes that share a row
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}

// lanes that differ in bits [log2 FROM, log2 TO) of their index end with the
// same sum: register moves only (DPP inside 16 lanes, the gfx950 half swaps
// beyond), 2 instructions per step where a shuffle through LDS takes a round
// trip
template <int FROM, int TO>
__device__ __forceinline__ float lane_sum(float v) {
  if constexpr (FROM <= 1 && TO > 1) v = dpp_add<0xB1>(v);      // quad_perm [1,0,3,2]
  if constexpr (FROM <= 2 && TO > 2) v = dpp_add<0x4E>(v);      // quad_perm [2,3,0,1]
  if constexpr (FROM <= 4 && TO > 4) {
    static_assert(FROM == 1, "the mirror below needs equal quads");
    v = dpp_add<0x141>(v);                                      // row_half_mirror: the other quad of 8
  }
  if constexpr (FROM <= 8 && TO > 8) v = dpp_add<0x128>(v);     // row_ror:8
  if constexpr (FROM <= 16 && TO > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (FROM <= 32 && TO > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Sum over the waves of one row: each wave has left its own sum in slot[wave]
// before a barrier.  One LDS read and log2(W) register steps.
template <int W>
__device__ __forceinline__ float waves_sum(const float* slot) {
  return lane_sum<1, W>(slot[threadIdx.x % W]);
}

// ---------------------------------------------------------------------------
// rows kept in registers
// ---------------------------------------------------------------------------
// LANES lanes share a row and hold NV chunks each: lane l the chunks l, l +
// LANES, ...; a workgroup of THREADS works on THREADS / LANES rows at a time.
template <int LANES, int THREADS>
struct Team {
  static constexpr int ROWS = THREADS / LANES;               // at a time
  static constexpr int WAVES = LANES > 64 ? LANES / 64 : 1;  // of one row
  static constexpr int SHARE = LANES < 64 ? LANES : 64;      // lanes of one wave that hold one row
  // which of the rows: the same for a whole wave where it can be, and then in
  // scalar registers, as are the row's addresses
  static __device__ __forceinline__ int index() {
    const int i = threadIdx.x / LANES;
    return LANES >= 64 ? __builtin_amdgcn_readfirstlane(i) : i;
  }
};

enum { PLAIN = 0, RESIDUAL = 1, DROPPED = 2 };

// Forward: one row per team, HBM bound: RMS norm of 8192 x 4096 bf16 20.3 us (6.6
// TB/s, a copy's rate), of 32768 x 4096 85 us (6.3); with residual and dropout,
// 131072 x 768 135 us (5.9).  Every load of the row goes out at once; the
// statistics are two sums over registers (mean, then squares about it).  One
// short-lived workgroup per few rows measured faster than workgroups that stay,
// hold the weights and fetch ahead (8192 x 4096 bf16 RMS norm, 25.8 us at the
// best grid against 24.9 us): few registers, so more waves and their loads in
// flight.  SAME: weight and bias are of the rows' type and are loaded as they are
// with the row; else they are widened after the sums (1-7% slower).
template <typename T, int LANES, int NV, int THREADS, int MODE, bool SAME>
__global__ __launch_bounds__(THREADS) void k_norm_fwd(FwdArgs a) {
  typedef typename T::raw raw;
  typedef Team<LANES, THREADS> G;
  constexpr int W = G::WAVES;
  __shared__ float red[2][G::ROWS][W];
  const int lane = threadIdx.x % LANES, grp = G::index(), wave = lane / 64;
  const int64_t row = a.first_row + (int64_t)blockIdx.x * G::ROWS + grp;
  const bool live = row < a.rows;
  const DropKey key = MODE == DROPPED ? drop_key(a.drop) : DropKey{};

  int col[NV], cnt[NV];
  Chunk<T> x[NV], res[NV], w[NV], b[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    col[v] = (lane + v * LANES) * 8;
    if (!live) col[v] = max(col[v], a.cols);
    cnt[v] = a.cols - col[v];
    x[v] = load_part<T>((const raw*)a.x + row * a.x_ld, col[v], a.cols);
    if constexpr (MODE != PLAIN) res[v] = load_part<T>((const raw*)a.residual + row * a.residual_ld, col[v], a.cols);
  }
  if constexpr (SAME) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      w[v] = load_part<T>((const raw*)a.weight, a.weight ? col[v] : a.cols, a.cols);
      b[v] = load_part<T>((const raw*)a.bias, a.bias ? col[v] : a.cols, a.cols);
    }
  }
  if (a.cols % 8)
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      settle_part<T>(x[v], col[v], a.cols);
      if constexpr (MODE != PLAIN) settle_part<T>(res[v], col[v], a.cols);
      if constexpr (SAME) {
        settle_part<T>(w[v], col[v], a.cols);
        settle_part<T>(b[v], col[v], a.cols);
      }
    }

  float s = 0.0f, q = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (MODE != PLAIN) {
      x[v] = join<T>(x[v], res[v], MODE == DROPPED, a.drop, key,
                     (uint64_t)row * (uint64_t)chunks_of(a.cols) + (uint64_t)(lane + v * LANES));
      if (cnt[v] > 0) store_chunk<T>((raw*)a.h + row * a.cols + col[v], x[v], cnt[v]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {                  // 0 past the row's end
      const float f = elem<T>(x[v], j);
      if (a.rms) { const float t = f * a.square_scale; q = fmaf(t, t, q); }
      else s = fmaf(f, a.sum_scale, s);
    }
  }
  float mean = 0.0f;
  if (!a.rms) {
    s = lane_sum<1, G::SHARE>(s);
    if constexpr (W > 1) {
      if ((lane & 63) == 0) red[0][grp][wave] = s;
      __syncthreads();
      s = waves_sum<W>(red[0][grp]);
    }
    mean = s * a.mean_scale;
    const float shift = -mean * a.square_scale;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = j < cnt[v] ? fmaf(elem<T>(x[v], j), a.square_scale, shift) : 0.0f;
        q = fmaf(t, t, q);
      }
  }
  q = lane_sum<1, G::SHARE>(q);
  if constexpr (W > 1) {
    if ((lane & 63) == 0) red[1][grp][wave] = q;
    __syncthreads();
    q = waves_sum<W>(red[1][grp]);
  }
  const float rstd = rsqrt_of(q * a.mean_scale + a.eps);
  if (live && lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (cnt[v] <= 0) continue;
    float f[8], pw[8], pb[8];
    if constexpr (SAME) {
#pragma unroll
      for (int j = 0; j < 8; ++j) { pw[j] = a.weight ? elem<T>(w[v], j) : 1.0f; pb[j] = elem<T>(b[v], j); }
    } else {
      load_param(a.weight, a.wdtype, col[v], cnt[v], 1.0f, pw);
      load_param(a.bias, a.wdtype, col[v], cnt[v], 0.0f, pb);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = fmaf((elem<T>(x[v], j) - mean) * rstd, pw[j], pb[j]);
    store_chunk<T>((raw*)a.y + row * a.cols + col[v], to_chunk<T>(f), cnt[v]);
  }
}

// Backward, weight gradients included: workgroups walk over the matrix, every
// lane adds up dy u and dy of its own columns over the rows its team meets, the
// teams of a workgroup add theirs through LDS at the end, and k_norm_bwd_reduce
// adds the workgroups'.  One pass over h, dy and dh, HBM bound: RMS norm of 8192 x
// 4096 bf16 34.2 us and 3.9 for the last sums, of 131072 x 768 102 us (5.9 TB/s);
// with dh and dropout 190-209 us from card to card (5.3-4.8 TB/s; arithmetic bounds it
// there: 350 instructions per chunk, 20 of them the generator's quarter-rate
// products, on lanes of which 768 columns leave a quarter idle).
//
// One chunk per lane and one workgroup of 16 waves on each compute unit: a second
// chunk costs 24 registers and drops the waves to 8, and twice the workgroups
// write twice the partial sums (8192 x 4096 bf16 RMS norm, sums included and with
// the caches full of other data: 42.8 us; two chunks per lane 53.0, 512 workgroups
// of half the size 52.3).  32 lanes of three chunks, which leave none idle at 768
// columns, have no registers for it (131072 rows with dropout, last sums included,
// 449 us against 193).  AHEAD: the next rows' loads go out before the current ones
// are worked on (188 us against 201 in one session); two rows ahead gain nothing
// more.  With two chunks per lane, the widest rows, registers do not allow it.
template <typename T, int LANES, int NV, int THREADS, int MODE>
__global__ __launch_bounds__(THREADS) void k_norm_bwd(BwdArgs a) {
  typedef typename T::raw raw;
  typedef Team<LANES, THREADS> G;
  constexpr int W = G::WAVES;
  constexpr bool AHEAD = NV == 1;
  __shared__ float red[2][2][G::ROWS][W];                    // used in turn, so one barrier per row is enough
  const int lane = threadIdx.x % LANES, grp = G::index(), wave = lane / 64;
  const DropKey key = MODE == DROPPED ? drop_key(a.drop) : DropKey{};

  int col[NV], cnt[NV];
  float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    col[v] = (lane + v * LANES) * 8;
    cnt[v] = a.cols - col[v];
#pragma unroll
    for (int j = 0; j < 8; ++j) { w[v][j] = 0.0f; dw[v][j] = 0.0f; db[v][j] = 0.0f; }
  }

  struct Row { Chunk<T> h[NV], dy[NV], dh[NV]; float mean, rstd; };
  auto fetch = [&](int64_t row, Row& r) {
    const bool live = row < a.rows;
    r.mean = live && !a.rms ? a.mean[row] : 0.0f;
    r.rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = live ? col[v] : a.cols;
      r.h[v] = load_part<T>((const raw*)a.h + row * a.h_ld, c, a.cols);
      r.dy[v] = load_part<T>((const raw*)a.dy + row * a.dy_ld, c, a.cols);
      if constexpr (MODE != PLAIN) r.dh[v] = load_part<T>((const raw*)a.dh + row * a.dh_ld, a.dh ? c : a.cols, a.cols);
    }
  };
  auto settle = [&](Row& r) {
    if (a.cols % 8)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        settle_part<T>(r.h[v], col[v], a.cols);
        settle_part<T>(r.dy[v], col[v], a.cols);
        if constexpr (MODE != PLAIN) settle_part<T>(r.dh[v], col[v], a.cols);
      }
  };

  int phase = 0;
  const int64_t step = (int64_t)gridDim.x * G::ROWS;
  int64_t row = (int64_t)blockIdx.x * G::ROWS + grp;
  Row next;
  if constexpr (AHEAD) fetch(row, next);
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (cnt[v] > 0) load_param(a.weight, a.wdtype, col[v], cnt[v], 1.0f, w[v]);
  for (int64_t first = (int64_t)blockIdx.x * G::ROWS; first < a.rows; first += step, row += step) {
    Row cur;
    if constexpr (AHEAD) {
      cur = next;
      if (first + step < a.rows) fetch(row + step, next);
    } else {
      fetch(row, cur);
    }
    settle(cur);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // past the row's end dy and w are 0 and u is some finite number of a finite row
        const float u = (elem<T>(cur.h[v], j) - cur.mean) * cur.rstd, dy = elem<T>(cur.dy[v], j), g = dy * w[v][j];
        s1 += g;
        s2 = fmaf(g, u, s2);
        dw[v][j] = fmaf(dy, u, dw[v][j]);
        db[v][j] += dy;
      }
    if (!(a.d || a.dx)) continue;                   // weight gradients alone
    s1 = lane_sum<1, G::SHARE>(s1);
    s2 = lane_sum<1, G::SHARE>(s2);
    if constexpr (W > 1) {
      if ((lane & 63) == 0) { red[phase][0][grp][wave] = s1; red[phase][1][grp][wave] = s2; }
      __syncthreads();
      s1 = waves_sum<W>(red[phase][0][grp]);
      s2 = waves_sum<W>(red[phase][1][grp]);
      phase ^= 1;
    }
    s1 = a.rms ? 0.0f : s1 * a.inv_cols;
    s2 *= -a.inv_cols;
    if (row >= a.rows) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (cnt[v] <= 0) continue;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = (elem<T>(cur.h[v], j) - cur.mean) * cur.rstd;
        const float t = fmaf(u, s2, elem<T>(cur.dy[v], j) * w[v][j] - s1);
        if constexpr (MODE != PLAIN) f[j] = fmaf(t, cur.rstd, elem<T>(cur.dh[v], j));
        else f[j] = t * cur.rstd;
      }
      if (a.d) store_chunk<T>((raw*)a.d + row * a.cols + col[v], to_chunk<T>(f), cnt[v]);
      if constexpr (MODE == DROPPED) {
        if (a.dx) {
          drop_chunk(a.drop, key, (uint64_t)row * (uint64_t)chunks_of(a.cols) + (uint64_t)(lane + v * LANES), f);
          store_chunk<T>((raw*)a.dx + row * a.cols + col[v], to_chunk<T>(f), cnt[v]);
        }
      }
    }
  }
  if (!a.partial) return;

  // the workgroup's sums: lanes of a wave that hold the same columns first
  // (teams smaller than a wave), then the waves (or teams) through LDS
  constexpr int PARTS = LANES < 64 ? THREADS / 64 : G::ROWS;
  constexpr int COLS = LANES * 8;                            // columns of one v
  if constexpr (PARTS == 1) {
    float* out = a.partial + (int64_t)blockIdx.x * a.cols;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (cnt[v] > 0) {
        store_chunk<F32>(out + col[v], to_chunk<F32>(dw[v]), cnt[v]);
        store_chunk<F32>(out + (int64_t)a.splits * a.cols + col[v], to_chunk<F32>(db[v]), cnt[v]);
      }
  } else {
    __shared__ float sum[PARTS][COLS];
    const int part = LANES < 64 ? threadIdx.x / 64 : grp;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float f = which ? db[v][j] : dw[v][j];
          f = lane_sum<G::SHARE, 64>(f);
          if (LANES >= 64 || (threadIdx.x & 63) < LANES) sum[part][lane * 8 + j] = f;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < COLS; c += THREADS) {
          float f = 0.0f;
#pragma unroll
          for (int i = 0; i < PARTS; ++i) f += sum[i][c];
          const int at = v * LANES * 8 + c;
          if (at < a.cols) a.partial[((int64_t)which * a.splits + blockIdx.x) * a.cols + at] = f;
        }
      }
  }
}

// One workgroup per row, the row read once per pass (from cache after the first):
// rows of any length.  838 x 20000 bf16 layer norm 27.2 us (2.5 TB/s), with a
// residual 39.8: a workgroup's 256 lanes wait for one chunk each per pass.
template <typename T>
__global__ __launch_bounds__(BLOCK) void k_norm_fwd_long(FwdArgs a) {
  __shared__ float red[BLOCK / 64];
  typedef typename T::raw raw;
  const DropKey key = drop_key(a.drop);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const raw* src = a.residual ? (const raw*)a.h + row * a.cols : (const raw*)a.x + row * a.x_ld;
    float s = 0.0f;
    for (int c0 = threadIdx.x * 8; c0 < a.cols; c0 += BLOCK * 8) {
      const int cnt = a.cols - c0;
      Chunk<T> c = load_chunk<T>((const raw*)a.x + row * a.x_ld + c0, cnt);
      if (a.residual) {
        const Chunk<T> res = load_chunk<T>((const raw*)a.residual + row * a.residual_ld + c0, cnt);
        c = join<T>(c, res, a.dropping, a.drop, key, (uint64_t)row * (uint64_t)chunks_of(a.cols) + (uint64_t)(c0 >> 3));
        store_chunk<T, true>((raw*)a.h + row * a.cols + c0, c, cnt);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cnt) {
          const float f = elem<T>(c, j), t = f * a.square_scale;
          s += a.rms ? t * t : f * a.sum_scale;
        }
    }
    s = block_sum<BLOCK>(s, red) * a.mean_scale;
    float mean = 0.0f, var = s;
    if (!a.rms) {
      mean = s;
      const float shift = -mean * a.square_scale;
      float q = 0.0f;
      for (int c0 = threadIdx.x * 8; c0 < a.cols; c0 += BLOCK * 8) {
        const int cnt = a.cols - c0;
        const Chunk<T> c = load_chunk<T>(src + c0, cnt);       // this thread's own stores, or x
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < cnt) { const float t = fmaf(elem<T>(c, j), a.square_scale, shift); q += t * t; }
      }
      var = block_sum<BLOCK>(q, red) * a.mean_scale;
    }
    const float rstd = rsqrt_of(var + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int c0 = threadIdx.x * 8; c0 < a.cols; c0 += BLOCK * 8) {
      const int cnt = a.cols - c0;
      const Chunk<T> c = load_chunk<T>(src + c0, cnt);
      float w[8], b[8], f[8];
      load_param(a.weight, a.wdtype, c0, cnt, 1.0f, w);
      load_param(a.bias, a.wdtype, c0, cnt, 0.0f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf((elem<T>(c, j) - mean) * rstd, w[j], b[j]);
      store_chunk<T>((raw*)a.y + row * a.cols + c0, to_chunk<T>(f), cnt);
    }
  }
}

// Gradients of the rows: one workgroup per row, two passes over it (838 x 20000
// bf16 layer norm 28.0 us).
template <typename T>
__global__ __launch_bounds__(BLOCK) void k_norm_bwd_rows_long(BwdArgs a) {
  __shared__ float red[BLOCK / 64];
  typedef typename T::raw raw;
  const DropKey key = drop_key(a.drop);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float mean = a.rms ? 0.0f : a.mean[row], rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c0 = threadIdx.x * 8; c0 < a.cols; c0 += BLOCK * 8) {
      const int cnt = a.cols - c0;
      const Chunk<T> h = load_chunk<T>((const raw*)a.h + row * a.h_ld + c0, cnt);
      const Chunk<T> dy = load_chunk<T>((const raw*)a.dy + row * a.dy_ld + c0, cnt);
      float w[8];
      load_param(a.weight, a.wdtype, c0, cnt, 1.0f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cnt) {
          const float g = elem<T>(dy, j) * w[j];
          s1 += g;
          s2 += g * ((elem<T>(h, j) - mean) * rstd);
        }
    }
    s1 = a.rms ? 0.0f : block_sum<BLOCK>(s1, red) * a.inv_cols;
    s2 = block_sum<BLOCK>(s2, red) * a.inv_cols;
    for (int c0 = threadIdx.x * 8; c0 < a.cols; c0 += BLOCK * 8) {
      const int cnt = a.cols - c0;
      const Chunk<T> h = load_chunk<T>((const raw*)a.h + row * a.h_ld + c0, cnt);
      const Chunk<T> dy = load_chunk<T>((const raw*)a.dy + row * a.dy_ld + c0, cnt);
      float w[8], f[8];
      load_param(a.weight, a.wdtype, c0, cnt, 1.0f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = (elem<T>(h, j) - mean) * rstd;
        f[j] = (elem<T>(dy, j) * w[j] - s1 - u * s2) * rstd;
      }
      if (a.dh) {
        const Chunk<T> dh = load_chunk<T>((const raw*)a.dh + row * a.dh_ld + c0, cnt);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += elem<T>(dh, j);
      }
      if (a.d) store_chunk<T>((raw*)a.d + row * a.cols + c0, to_chunk<T>(f), cnt);
      if (a.dx) {
        drop_chunk(a.drop, key, (uint64_t)row * (uint64_t)chunks_of(a.cols) + (uint64_t)(c0 >> 3), f);
        store_chunk<T>((raw*)a.dx + row * a.cols + c0, to_chunk<T>(f), cnt);
      }
    }
  }
}

// Gradients of weight and bias: workgroup (bx, by) sums 32 chunks of columns
// over the rows r = by * 8 + lane row (mod 8 * splits) and writes one partial
// sum per column (838 x 20000 bf16 layer norm 13.4 us).  The wider the rows the
// fewer the ranges of rows, so a lane adds up LONG_TERMS rows at a time and then
// those sums: one chain over all its rows would be rows / 8 long past 262144
// columns (200003 equal rows of 262408: relative errors to 3.7e-4, against 5.9e-6).
constexpr int LONG_TERMS = 64;

template <typename T>
__global__ __launch_bounds__(BLOCK) void k_norm_bwd_cols_long(BwdArgs a) {
  typedef typename T::raw raw;
  __shared__ float sw[8][256], sb[8][256];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c0 = (blockIdx.x * 32 + lane) * 8, cnt = a.cols - c0;
  float dw[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.0f;
  for (int64_t row = (int64_t)blockIdx.y * 8 + grp; cnt > 0 && row < a.rows;) {
    float pw[8], pb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) pw[j] = pb[j] = 0.0f;
    for (int term = 0; term < LONG_TERMS && row < a.rows; ++term, row += (int64_t)a.splits * 8) {
      const float mean = a.rms ? 0.0f : a.mean[row], rstd = a.rstd[row];
      const Chunk<T> h = load_chunk<T>((const raw*)a.h + row * a.h_ld + c0, cnt);
      const Chunk<T> dy = load_chunk<T>((const raw*)a.dy + row * a.dy_ld + c0, cnt);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = elem<T>(dy, j);
        pw[j] += g * ((elem<T>(h, j) - mean) * rstd);
        pb[j] += g;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) { dw[j] += pw[j]; db[j] += pb[j]; }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) { sw[grp][lane * 8 + j] = dw[j]; sb[grp][lane * 8 + j] = db[j]; }
  __syncthreads();
  const int col = blockIdx.x * 256 + threadIdx.x;
  float tw = 0.0f, tb = 0.0f;
#pragma unroll
  for (int g = 0; g < 8; ++g) { tw += sw[g][threadIdx.x]; tb += sb[g][threadIdx.x]; }
  if (col < a.cols) {
    a.partial[(int64_t)blockIdx.y * a.cols + col] = tw;
    a.partial[((int64_t)a.splits + blockIdx.y) * a.cols + col] = tb;
  }
}

// dw, db = the partial sums over `splits` (0 of them: zeros), in a fixed order.  A
// launch's latency and one memory round trip: 3.9 us for 256 x 4096.
struct ReduceArgs {
  const float* partial;
  void *dweight, *dbias;
  int cols, splits, wdtype;
};

__global__ __launch_bounds__(1024) void k_norm_bwd_reduce(ReduceArgs a) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  void* out = blockIdx.y ? a.dbias : a.dweight;
  if (!out) return;
  const float* src = a.partial + (int64_t)blockIdx.y * a.splits * a.cols;
  float s = 0.0f;
  if (col < a.cols)
    for (int first = grp; first < a.splits; first += 32 * 8) {
      float f[8];                                   // loads of one turn go out together
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = first + 32 * k;
        f[k] = i < a.splits ? ((const FO_GLB float*)src)[(int64_t)i * a.cols + col] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s += f[k];
    }
  part[grp][lane] = s;
  __syncthreads();
#pragma unroll
  for (int step = 16; step; step >>= 1) {
    if (grp < step) part[grp][lane] += part[grp + step][lane];
    __syncthreads();
  }
  if (grp == 0 && col < a.cols) store_param(out, a.wdtype, col, part[0][lane]);
}

}  // namespace rows
}  // namespace fo
