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
  int64_t rows, x_ld;
  int cols;
  DropArgs drop;
};

struct FwdArgs {
  const void *x, *residual, *weight, *bias;
  void *h, *y;
  float *mean, *rstd;
  int64_t rows, x_ld, residual_ld;
  int cols, wdtype, rms, dropping;
  float eps, inv_cols;
  DropArgs drop;
};

struct BwdArgs {
  const void *dy, *dh, *h, *weight;
  const float *mean, *rstd;
  void *d, *dx;
  float* partial;              // [2][splits][cols]: dw, db
  int64_t rows, dy_ld, dh_ld, h_ld;
  int cols, wdtype, rms, dropping, splits;
  float inv_cols;
  DropArgs drop;
};

__device__ __forceinline__ int chunks_of(int cols) { return (cols + 7) >> 3; }

// ---------------------------------------------------------------------------
// dropout (the gradient is the same call on the output's gradient)
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(BLOCK) void k_dropout(DropoutArgs a) {
  const int nch = chunks_of(a.cols);
  const int64_t total = a.rows * nch;
  const DropKey key = drop_key(a.drop);
  for (int64_t i = (int64_t)blockIdx.x * BLOCK + threadIdx.x; i < total; i += (int64_t)gridDim.x * BLOCK) {
    const int64_t r = i / nch;
    const int c0 = (int)(i - r * nch) * 8, cnt = a.cols - c0;
    const Chunk<T> in = load_chunk<T>((const typename T::raw*)a.x + r * a.x_ld + c0, cnt);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = elem<T>(in, j) * a.drop.scale;
    if (a.drop.all) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    } else {
      drop_chunk(a.drop, key, (uint64_t)i, f);
    }
    store_chunk<T>((typename T::raw*)a.y + r * (int64_t)a.cols + c0, to_chunk<T>(f), cnt);
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
__device__ __forceinline__ Chunk<T> join_chunk(const FwdArgs& a, const DropKey& key, int64_t row, int c0, int cnt,
                                               const Chunk<T>& x) {
  const Chunk<T> res = load_chunk<T>((const typename T::raw*)a.residual + row * a.residual_ld + c0, cnt);
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = elem<T>(x, j);
  if (a.dropping) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= a.drop.scale;
    if (a.drop.all) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    } else {
      drop_chunk(a.drop, key, (uint64_t)row * (uint64_t)chunks_of(a.cols) + (uint64_t)(c0 >> 3), f);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] += elem<T>(res, j);
  return to_chunk<T>(f);
}

// One workgroup per row, the row read once per pass: rows of any length.
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
        c = join_chunk<T>(a, key, row, c0, cnt, c);
        store_chunk<T>((raw*)a.h + row * a.cols + c0, c, cnt);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cnt) s += a.rms ? elem<T>(c, j) * elem<T>(c, j) : elem<T>(c, j);
    }
    s = block_sum<BLOCK>(s, red) * a.inv_cols;
    float mean = 0.0f, var = s;
    if (!a.rms) {
      mean = s;
      float q = 0.0f;
      for (int c0 = threadIdx.x * 8; c0 < a.cols; c0 += BLOCK * 8) {
        const int cnt = a.cols - c0;
        const Chunk<T> c = load_chunk<T>(src + c0, cnt);       // this thread's own stores, or x
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < cnt) { const float t = elem<T>(c, j) - mean; q += t * t; }
      }
      var = block_sum<BLOCK>(q, red) * a.inv_cols;
    }
    const float rstd = 1.0f / sqrtf(var + a.eps);
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

// Gradients of the rows: one workgroup per row, two passes over it.
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
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= a.drop.scale;
        if (a.drop.all) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = 0.0f;
        } else {
          drop_chunk(a.drop, key, (uint64_t)row * (uint64_t)chunks_of(a.cols) + (uint64_t)(c0 >> 3), f);
        }
        store_chunk<T>((raw*)a.dx + row * a.cols + c0, to_chunk<T>(f), cnt);
      }
    }
  }
}

// Gradients of weight and bias: workgroup (bx, by) sums 32 chunks of columns
// over the rows r = by * 8 + lane row (mod 8 * splits) and writes one partial
// sum per column.
template <typename T>
__global__ __launch_bounds__(BLOCK) void k_norm_bwd_cols_long(BwdArgs a) {
  typedef typename T::raw raw;
  __shared__ float sw[8][256], sb[8][256];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c0 = (blockIdx.x * 32 + lane) * 8, cnt = a.cols - c0;
  float dw[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.0f;
  if (cnt > 0)
    for (int64_t row = (int64_t)blockIdx.y * 8 + grp; row < a.rows; row += (int64_t)a.splits * 8) {
      const float mean = a.rms ? 0.0f : a.mean[row], rstd = a.rstd[row];
      const Chunk<T> h = load_chunk<T>((const raw*)a.h + row * a.h_ld + c0, cnt);
      const Chunk<T> dy = load_chunk<T>((const raw*)a.dy + row * a.dy_ld + c0, cnt);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = elem<T>(dy, j);
        dw[j] += g * ((elem<T>(h, j) - mean) * rstd);
        db[j] += g;
      }
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

// dw, db = the partial sums over `splits` (0 of them: zeros), in a fixed order
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
    for (int i = grp; i < a.splits; i += 32) s += ((const FO_GLB float*)src)[(int64_t)i * a.cols + col];
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
