// fo_rows.hip -- C ABI of the row operators (dropout, layer norm, RMS norm and
// their fused form; see include/foamd.h for the contract of every entry
// point).  Host work is argument validation and launches; nothing here
// allocates, synchronises, keeps state between calls or throws.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/foamd.h"
#include "fo_error.hpp"
#include "fo_rows_args.hpp"
#include "fo_rows_kernels.hpp"

using namespace fo;
using namespace fo::rows;

namespace {

constexpr int64_t kMaxThreads = int64_t(1) << 31;  // of one launch (a grid's threads must fit 32 bits)

#define FO_TRY(expr) do { const int rc_ = (expr); if (rc_) return rc_; } while (0)

int drop_args(const fo_dropout_key* key, DropArgs* d) {
  if (!(key->p >= 0.0 && key->p <= 1.0)) return fail(FO_EINVAL, "the drop probability must lie in [0, 1]");
  if (reinterpret_cast<uintptr_t>(key->state) % 8) return fail(FO_EINVAL, "key.state is not 8-byte aligned");
  const double two32 = 4294967296.0, t = std::nearbyint(key->p * two32);
  d->all = t >= two32;
  d->thr = d->all ? 0xffffffffu : (uint32_t)t;
  d->scale = d->all ? 0.0f : (float)(two32 / (two32 - t));
  d->seed = key->seed;
  d->offset = key->offset;
  d->state = key->state;
  return FO_OK;
}

int launch_check(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FO_OK : fail(FO_EHIP, "%s: %s", what, hipGetErrorString(e));
}

// workgroups of BLOCK threads for kernels that loop over what they do not cover
unsigned grid_of(int64_t want) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(want, kMaxThreads / BLOCK)); }

#define FO_BY_TYPE(dtype, KERNEL, ...)                                     \
  do {                                                                     \
    if ((dtype) == FO_BF16) hipLaunchKernelGGL(KERNEL<Bf16>, __VA_ARGS__); \
    else if ((dtype) == FO_FP16) hipLaunchKernelGGL(KERNEL<Fp16>, __VA_ARGS__); \
    else hipLaunchKernelGGL(KERNEL<F32>, __VA_ARGS__);                     \
  } while (0)

template <bool FLAT, typename Index>
void drop_launch(int dtype, unsigned groups, const DropoutArgs& a, hipStream_t s) {
  if (dtype == FO_BF16) hipLaunchKernelGGL((k_dropout<Bf16, FLAT, Index>), groups, BLOCK, 0, s, a);
  else if (dtype == FO_FP16) hipLaunchKernelGGL((k_dropout<Fp16, FLAT, Index>), groups, BLOCK, 0, s, a);
  else hipLaunchKernelGGL((k_dropout<F32, FLAT, Index>), groups, BLOCK, 0, s, a);
}

template <typename T, int LANES, int NV, int MODE, bool SAME>
void launch_fwd(FwdArgs a, hipStream_t s) {
  constexpr int threads = fwd_threads(LANES), at_a_time = threads / LANES;
  constexpr int64_t most = kMaxThreads / threads;             // workgroups of one launch
  const int64_t groups = (a.rows + at_a_time - 1) / at_a_time;
  for (int64_t g = 0; g < groups; g += most) {
    a.first_row = g * at_a_time;
    hipLaunchKernelGGL((k_norm_fwd<T, LANES, NV, threads, MODE, SAME>), (unsigned)std::min(groups - g, most), threads, 0,
                       s, a);
  }
}

template <typename T, int LANES, int NV>
void fwd_mode(int mode, bool same, const FwdArgs& a, hipStream_t s) {
  if (same) {
    if (mode == PLAIN) launch_fwd<T, LANES, NV, PLAIN, true>(a, s);
    else if (mode == RESIDUAL) launch_fwd<T, LANES, NV, RESIDUAL, true>(a, s);
    else launch_fwd<T, LANES, NV, DROPPED, true>(a, s);
  } else {
    if (mode == PLAIN) launch_fwd<T, LANES, NV, PLAIN, false>(a, s);
    else if (mode == RESIDUAL) launch_fwd<T, LANES, NV, RESIDUAL, false>(a, s);
    else launch_fwd<T, LANES, NV, DROPPED, false>(a, s);
  }
}

template <typename T>
void fwd_type(Spread sp, int mode, bool same, const FwdArgs& a, hipStream_t s) {
  switch (sp.lanes) {
    case 8: return sp.chunks == 1 ? fwd_mode<T, 8, 1>(mode, same, a, s) : fwd_mode<T, 8, 2>(mode, same, a, s);
    case 16: return fwd_mode<T, 16, 2>(mode, same, a, s);
    case 32: return sp.chunks == 3 ? fwd_mode<T, 32, 3>(mode, same, a, s) : fwd_mode<T, 32, 2>(mode, same, a, s);
    case 64: return fwd_mode<T, 64, 2>(mode, same, a, s);
    case 128: return fwd_mode<T, 128, 2>(mode, same, a, s);
    case 256: return fwd_mode<T, 256, 2>(mode, same, a, s);
    case 512: return fwd_mode<T, 512, 2>(mode, same, a, s);
    // two workgroups of 1024 fit a compute unit up to 64 registers: with dropout not
    // next to weights loaded up front (1024 x 16384 bf16, 29.2 us against 34.6)
    default: return fwd_mode<T, 1024, 2>(mode, same && mode != DROPPED, a, s);
  }
}

template <typename T, int LANES, int NV, int MODE>
void launch_bwd(const BwdArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_norm_bwd<T, LANES, NV, kBwdThreads, MODE>), (unsigned)a.splits, kBwdThreads, 0, s, a);
}

template <typename T, int LANES>
void bwd_mode(int mode, const BwdArgs& a, hipStream_t s) {
  if (mode == PLAIN) launch_bwd<T, LANES, 1, PLAIN>(a, s);
  else if (mode == RESIDUAL) launch_bwd<T, LANES, 1, RESIDUAL>(a, s);
  else launch_bwd<T, LANES, 1, DROPPED>(a, s);
}

template <typename T>
void bwd_type(Spread sp, int mode, const BwdArgs& a, hipStream_t s) {
  if constexpr (!is_f32<T>)
    if (sp.chunks == 2) return mode == PLAIN ? launch_bwd<T, 1024, 2, PLAIN>(a, s) : launch_bwd<T, 1024, 2, RESIDUAL>(a, s);
  switch (sp.lanes) {
    case 8: return bwd_mode<T, 8>(mode, a, s);
    case 16: return bwd_mode<T, 16>(mode, a, s);
    case 32: return bwd_mode<T, 32>(mode, a, s);
    case 64: return bwd_mode<T, 64>(mode, a, s);
    case 128: return bwd_mode<T, 128>(mode, a, s);
    case 256: return bwd_mode<T, 256>(mode, a, s);
    case 512: return bwd_mode<T, 512>(mode, a, s);
    default: return bwd_mode<T, 1024>(mode, a, s);
  }
}

}  // namespace

extern "C" {

int fo_dropout(const void* x, int64_t x_ld, void* y, int64_t rows, int64_t cols, int dtype, const fo_dropout_key* key,
               void* stream) {
  clear_error();
  if (!key) return fail(FO_EINVAL, "key is NULL");
  if (!dtype_ok(dtype)) return fail(FO_EINVAL, "bad element type %d", dtype);
  if (rows == 0 || cols == 0) return rows < 0 || cols < 0 ? fail(FO_EINVAL, "negative size") : FO_OK;
  FO_TRY(drop_shape_ok(rows, cols));
  DropoutArgs a = {};
  FO_TRY(drop_args(key, &a.drop));
  Arrays ar;
  FO_TRY(ar.add(x, "x", false, true, rows, cols, x_ld, elem_size(dtype)));
  FO_TRY(ar.add(y, "y", true, true, rows, cols, cols, elem_size(dtype)));
  FO_TRY(ar.disjoint());
  a.x = x; a.y = y; a.rows = rows; a.x_ld = x_ld; a.cols = cols;
  const int64_t chunks = rows * ((cols + 7) / 8);
  const unsigned groups = grid_of((chunks + BLOCK * DROP_PER - 1) / (BLOCK * DROP_PER));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (cols % 8 == 0 && (x_ld == cols || rows == 1)) drop_launch<true, int64_t>(dtype, groups, a, s);
  else if (chunks < (int64_t(1) << 31) && cols <= kMaxCols) drop_launch<false, uint32_t>(dtype, groups, a, s);
  else drop_launch<false, int64_t>(dtype, groups, a, s);
  return launch_check("dropout launch");
}

int fo_norm_forward(const fo_norm_fwd* in, void* stream) {
  clear_error();
  if (!in) return fail(FO_EINVAL, "args is NULL");
  if (!dtype_ok(in->dtype) || !dtype_ok(in->wdtype)) return fail(FO_EINVAL, "bad element type");
  if (in->kind != FO_LAYER_NORM && in->kind != FO_RMS_NORM) return fail(FO_EINVAL, "bad norm kind %d", in->kind);
  FO_TRY(shape_ok(in->rows, in->cols));
  if (!(in->eps >= 0.0 && std::isfinite(in->eps))) return fail(FO_EINVAL, "eps must be finite and >= 0");
  const bool rms = in->kind == FO_RMS_NORM;
  if (rms && (in->bias || in->mean)) return fail(FO_EINVAL, "an RMS norm has no bias and no mean");
  FwdArgs a = {};
  FO_TRY(drop_args(&in->drop, &a.drop));
  a.dropping = a.drop.thr != 0;
  // (with no rows every array may be NULL: nothing is read or written)
  if (in->rows > 0 && !in->residual && (in->h || in->drop.p != 0.0))
    return fail(FO_EINVAL, "h and dropout need a residual");
  const int64_t rows = in->rows, cols = in->cols;
  const size_t es = elem_size(in->dtype), ws = elem_size(in->wdtype);
  const bool any = rows > 0;
  Arrays ar;
  FO_TRY(ar.add(in->x, "x", false, any, rows, cols, in->x_ld, es));
  FO_TRY(ar.add(in->residual, "residual", false, false, rows, cols, in->residual_ld, es));
  FO_TRY(ar.add(in->weight, "weight", false, false, 1, cols, 0, ws));
  FO_TRY(ar.add(in->bias, "bias", false, false, 1, cols, 0, ws));
  FO_TRY(ar.add(in->h, "h", true, any && in->residual, rows, cols, cols, es));
  FO_TRY(ar.add(in->y, "y", true, any, rows, cols, cols, es));
  FO_TRY(ar.add(in->mean, "mean", true, false, rows, 1, 1, 4));
  FO_TRY(ar.add(in->rstd, "rstd", true, false, rows, 1, 1, 4));
  FO_TRY(ar.disjoint());
  if (!any) return FO_OK;
  a.x = in->x; a.residual = in->residual; a.weight = in->weight; a.bias = in->bias;
  a.h = in->h; a.y = in->y; a.mean = in->mean; a.rstd = in->rstd;
  a.rows = rows; a.x_ld = in->x_ld; a.residual_ld = in->residual_ld;
  a.cols = (int)cols; a.wdtype = in->wdtype; a.rms = rms;
  const int k = quarter_log(cols);
  a.eps = (float)in->eps;
  a.sum_scale = std::ldexp(1.0f, -2 * k); a.square_scale = std::ldexp(1.0f, -k);
  a.mean_scale = std::ldexp((float)(1.0 / (double)cols), 2 * k);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int mode = !in->residual ? PLAIN : a.dropping ? DROPPED : RESIDUAL;
  const bool same = in->wdtype == in->dtype || (!in->weight && !in->bias);
  const Spread sp = fwd_spread(cols);
  if (!sp.lanes) FO_BY_TYPE(in->dtype, k_norm_fwd_long, grid_of(rows), BLOCK, 0, s, a);
  else if (in->dtype == FO_BF16) fwd_type<Bf16>(sp, mode, same, a, s);
  else if (in->dtype == FO_FP16) fwd_type<Fp16>(sp, mode, same, a, s);
  else fwd_type<F32>(sp, mode, same, a, s);
  return launch_check("norm forward launch");
}

int fo_norm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes) {
  clear_error();
  if (!bytes) return fail(FO_EINVAL, "bytes is NULL");
  FO_TRY(shape_ok(rows, cols));
  *bytes = bwd_workspace(rows, cols);
  return FO_OK;
}

int fo_norm_backward(const fo_norm_bwd* in, void* stream) {
  clear_error();
  if (!in) return fail(FO_EINVAL, "args is NULL");
  if (!dtype_ok(in->dtype) || !dtype_ok(in->wdtype)) return fail(FO_EINVAL, "bad element type");
  if (in->kind != FO_LAYER_NORM && in->kind != FO_RMS_NORM) return fail(FO_EINVAL, "bad norm kind %d", in->kind);
  FO_TRY(shape_ok(in->rows, in->cols));
  const bool rms = in->kind == FO_RMS_NORM;
  if (rms && (in->dbias || in->mean)) return fail(FO_EINVAL, "an RMS norm has no bias and no mean");
  BwdArgs a = {};
  FO_TRY(drop_args(&in->drop, &a.drop));
  if (in->dx && in->drop.p == 0.0) return fail(FO_EINVAL, "dx is for dropout: without it the gradient is d");
  const int64_t rows = in->rows, cols = in->cols;
  const size_t es = elem_size(in->dtype), ws = elem_size(in->wdtype);
  const bool any = rows > 0, params = in->dweight || in->dbias, grads = in->d || in->dx;
  const bool dropping = in->dx != nullptr;
  const int64_t splits = bwd_splits(rows, cols, in->dtype, dropping);
  Arrays ar;
  FO_TRY(ar.add(in->dy, "dy", false, any, rows, cols, in->dy_ld, es));
  FO_TRY(ar.add(in->dh, "dh", false, false, rows, cols, in->dh_ld, es));
  FO_TRY(ar.add(in->h, "h", false, any, rows, cols, in->h_ld, es));
  FO_TRY(ar.add(in->weight, "weight", false, false, 1, cols, 0, ws));
  FO_TRY(ar.add(in->mean, "mean", false, any && !rms, rows, 1, 1, 4));
  FO_TRY(ar.add(in->rstd, "rstd", false, any, rows, 1, 1, 4));
  FO_TRY(ar.add(in->d, "d", true, false, rows, cols, cols, es));
  FO_TRY(ar.add(in->dx, "dx", true, false, rows, cols, cols, es));
  FO_TRY(ar.add(in->dweight, "dweight", true, false, 1, cols, 0, ws));
  FO_TRY(ar.add(in->dbias, "dbias", true, false, 1, cols, 0, ws));
  if (params && any) {
    const int64_t need = 2 * splits * cols * (int64_t)sizeof(float);
    if (in->workspace_bytes < need)
      return fail(FO_EINVAL, "the workspace holds %lld bytes, %lld are needed", (long long)in->workspace_bytes,
                  (long long)need);
    FO_TRY(ar.add(in->workspace, "workspace", true, true, 1, need, 0, 1, 16));
  }
  FO_TRY(ar.disjoint());
  a.dy = in->dy; a.dh = in->dh; a.h = in->h; a.weight = in->weight; a.mean = in->mean; a.rstd = in->rstd;
  a.d = in->d; a.dx = in->dx; a.partial = params ? (float*)in->workspace : nullptr;
  a.rows = rows; a.dy_ld = in->dy_ld; a.dh_ld = in->dh_ld; a.h_ld = in->h_ld;
  a.cols = (int)cols; a.wdtype = in->wdtype; a.rms = rms; a.splits = (int)splits;
  a.inv_cols = (float)(1.0 / (double)cols);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Spread sp = bwd_spread(cols, in->dtype, dropping);
  if (any && sp.lanes) {
    const int mode = dropping ? DROPPED : in->dh ? RESIDUAL : PLAIN;
    if (!grads && !params) return FO_OK;
    if (in->dtype == FO_BF16) bwd_type<Bf16>(sp, mode, a, s);
    else if (in->dtype == FO_FP16) bwd_type<Fp16>(sp, mode, a, s);
    else bwd_type<F32>(sp, mode, a, s);
    FO_TRY(launch_check("norm backward launch"));
  } else if (any) {
    if (grads) FO_BY_TYPE(in->dtype, k_norm_bwd_rows_long, grid_of(rows), BLOCK, 0, s, a);
    if (params)
      FO_BY_TYPE(in->dtype, k_norm_bwd_cols_long, dim3((unsigned)((cols + 255) / 256), (unsigned)splits), BLOCK, 0, s, a);
    FO_TRY(launch_check("norm backward launch"));
  }
  if (params) {
    ReduceArgs r = {(const float*)in->workspace, in->dweight, in->dbias, (int)cols, any ? (int)splits : 0, in->wdtype};
    hipLaunchKernelGGL(k_norm_bwd_reduce, dim3((unsigned)((cols + 31) / 32), in->dbias ? 2 : 1), 1024, 0, s, r);
    FO_TRY(launch_check("weight gradient sum launch"));
  }
  return FO_OK;
}

}  // extern "C"
