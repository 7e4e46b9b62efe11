// fo_products.hip -- C ABI of the operators built on matrix products: linear cross
// entropy and the gated block (see include/foamd.h for the contract of every entry
// point).  Host work is argument validation and launches; nothing here allocates,
// synchronises, keeps state between calls or throws.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/foamd.h"
#include "fo_error.hpp"
#include "fo_products_args.hpp"
#include "fo_products_kernels.hpp"

using namespace fo;
using namespace fo::prod;
using rows::Arrays;

namespace {

#define FO_TRY(expr) do { const int rc_ = (expr); if (rc_) return rc_; } while (0)

int launch_check(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FO_OK : fail(FO_EHIP, "%s: %s", what, hipGetErrorString(e));
}

unsigned grid_of(int64_t want, int64_t most = 1 << 16) { return (unsigned)std::max<int64_t>(1, std::min(want, most)); }

template <typename T, typename E, Form F, TileKind K, int WR, int WC, int FR, int FC, int NS, int KS = 1>
void launch_tile(const Product& p, const typename E::Args& e, hipStream_t s) {
  static_assert(tile_r(K) == WR * FR * 32 && tile_c(K) == WC * FC * 32 && waves_r(K) == WR && threads(K) == WR * WC * KS * 64,
                "the tile is the one that sizes, workspaces and limits were worked out for");
  const unsigned groups = (unsigned)p.tiles_r * (unsigned)p.tiles_c * (unsigned)p.slices;
  hipLaunchKernelGGL((k_product<T, WR, WC, FR, FC, NS, KS, F, E>), groups, WR * WC * KS * 64, 0, s, p, e);
}

template <typename T, typename E, Form F>
void launch_product(Product p, const Cut& c, const typename E::Args& e, hipStream_t s) {
  p.tiles_r = c.tiles_r; p.tiles_c = c.tiles_c; p.slices = c.slices;
  if (c.kind == NARROW) {
    // three stages let four workgroups share a compute unit; where two do (512 tiles and
    // fewer) a fourth stage is more under way: one token through two 14336 x 4096 bf16
    // weights from memory 47.6 us against 49.5; six stages, or steps fetched in pairs,
    // gave no more.  786 tiles (50257 x 768) take 25 us with four stages, 18 with three.
    if ((int64_t)c.tiles_r * c.tiles_c * c.slices <= 2 * kUnits) return launch_tile<T, E, F, NARROW, 1, 1, 2, 1, 4>(p, e, s);
    return launch_tile<T, E, F, NARROW, 1, 1, 2, 1, 3>(p, e, s);
  }
  if (c.kind == WIDE) return launch_tile<T, E, F, WIDE, 2, 4, 4, 2, 2>(p, e, s);
  if (c.kind == MIDDLE) return launch_tile<T, E, F, MIDDLE, 2, 2, 2, 2, 2>(p, e, s);
  // two groups of two waves: with one, half of the matrix units idle where a tile is all that a
  // compute unit has (gated block of 100 x 768 x 2048 float32 34 us against 22, bf16 with
  // gradients 35 against 33; head of 100 x 768 x 5000 with gradients 113 against 89)
  launch_tile<T, E, F, SMALL, 1, 2, 2, 1, 4, 2>(p, e, s);
}

uint8_t* at(void* workspace, int64_t offset) { return offset < 0 ? nullptr : static_cast<uint8_t*>(workspace) + offset; }

// An operand as its product reads it: the caller's rows, or a copy in the workspace.
struct Operand { const void* p; int64_t ld; };

// The copies that a call needs, made by one launch.
struct Packing {
  int dtype;
  void* workspace;
  PackJobs jobs = {};
  int n = 0;
  int64_t most = 0;

  // rows x cols elements into dst_rows rows of `k` elements at `offset`
  Operand copy(const void* src, int64_t ld, int64_t rows, int64_t cols, int64_t offset, int64_t k, int64_t dst_rows,
               const int64_t* target = nullptr, int64_t ignore = 0) {
    const int64_t es = (int64_t)elem_size(dtype);
    jobs.job[n++] = {src, ld, at(workspace, offset), k, (int)rows, (int)cols, (int)dst_rows, target, ignore};
    most = std::max(most, dst_rows * k * es / 16);
    return {at(workspace, offset), k};
  }
  Operand operand(const void* src, int64_t ld, int64_t rows, int64_t cols, int64_t offset, int64_t k) {
    return offset < 0 ? Operand{src, ld} : copy(src, ld, rows, cols, offset, k, rows);
  }
  void launch(hipStream_t s) {
    if (!n) return;
    const dim3 groups(grid_of((most + 511) / 512), (unsigned)n);
    if (dtype == FO_F32) hipLaunchKernelGGL(k_pack<uint32_t>, groups, 256, 0, s, jobs);
    else hipLaunchKernelGGL(k_pack<uint16_t>, groups, 256, 0, s, jobs);
    n = 0;
    most = 0;
  }
};

Product product_of(const Operand& r, int64_t nr, const Operand& c, int64_t nc, int64_t k, int64_t es) {
  Product p = {};
  p.r = r.p; p.c = c.p;
  p.r_ld = r.ld * es; p.c_ld = c.ld * es;
  p.nr = (int)nr; p.nc = (int)nc;
  p.k = (int)k;
  p.steps = (int)((k * es + 127) / 128);
  return p;
}

// ---------------------------------------------------------------------------
// linear cross entropy
// ---------------------------------------------------------------------------
int area_check(int64_t rows, int64_t cols, int64_t out) {
  if (rows * cols > kMaxArea || rows * out > kMaxArea || cols * out > kMaxArea)
    return fail(FO_EINVAL, "the product of two of the sizes %lld, %lld and %lld is more than 2^36", (long long)rows,
                (long long)cols, (long long)out);
  return FO_OK;
}

int loss_checks(const fo_loss* a) {
  if (!a) return fail(FO_EINVAL, "args is NULL");
  if (!dtype_ok(a->dtype)) return fail(FO_EINVAL, "bad element type %d", a->dtype);
  if (a->reduction < FO_LOSS_NONE || a->reduction > FO_LOSS_SUM) return fail(FO_EINVAL, "bad reduction %d", a->reduction);
  if (a->rows < 0 || a->rows > kMaxTokens) return fail(FO_EINVAL, "rows = %lld is not in [0, 2^21]", (long long)a->rows);
  if (a->cols < 1 || a->cols > kMaxCols) return fail(FO_EINVAL, "cols = %lld is not in [1, 2^20]", (long long)a->cols);
  if (a->vocab < 1 || a->vocab > kMaxVocab) return fail(FO_EINVAL, "vocab = %lld is not in [1, 2^24]", (long long)a->vocab);
  FO_TRY(area_check(a->rows, a->cols, a->vocab));
  if (!(a->smoothing >= 0.0 && a->smoothing <= 1.0)) return fail(FO_EINVAL, "the smoothing must lie in [0, 1]");
  return FO_OK;
}

int loss_inputs(const fo_loss* a, Arrays& ar) {
  const size_t es = elem_size(a->dtype);
  const bool any = a->rows > 0;
  FO_TRY(ar.add(a->x, "x", false, any, a->rows, a->cols, a->x_ld, es));
  FO_TRY(ar.add(a->weight, "weight", false, any, a->vocab, a->cols, a->weight_ld, es));
  FO_TRY(ar.add(a->target, "target", false, any, a->rows, 1, 1, 8));
  return FO_OK;
}

int workspace_check(void* workspace, int64_t have, int64_t need, Arrays& ar) {
  if (!need) return FO_OK;
  if (have < need)
    return fail(FO_EINVAL, "the workspace holds %lld bytes, %lld are needed", (long long)have, (long long)need);
  return ar.add(workspace, "workspace", true, true, 1, need, 0, 1, 256);
}

void join_rows(LossRows r, hipStream_t s) {
  r.width = 1;
  while (r.width < 16 && r.width * 256 < r.rows) r.width *= 2;
  hipLaunchKernelGGL(k_loss_rows, (unsigned)((r.rows + r.width - 1) / r.width), 1024, 0, s, r);
}

template <typename T>
int run_loss_forward(const fo_loss* a, float* rest, const LossForward& f, hipStream_t s) {
  const int64_t es = elem_bytes<T>;
  Packing pack = {a->dtype, a->workspace};
  const Operand x = pack.operand(a->x, a->x_ld, a->rows, a->cols, f.x, f.k);
  const Operand w = pack.operand(a->weight, a->weight_ld, a->vocab, a->cols, f.w, f.k);
  pack.launch(s);
  const bool reduced = a->reduction != FO_LOSS_NONE;
  v2f* part = (v2f*)at(a->workspace, f.part);
  float* sums = (float*)at(a->workspace, f.sums);
  float* chosen = (float*)at(a->workspace, f.chosen);
  float* each = reduced ? (float*)at(a->workspace, f.each) : a->loss;
  const Product p = product_of(w, a->vocab, x, a->rows, f.k, es);
  launch_product<T, Statistics, ROWS_ROWS>(p, f.c, {part, sums, chosen, a->target, a->ignore_index}, s);
  join_rows({part, sums, chosen, a->target, each, a->lse, nullptr, rest, a->ignore_index, (int)a->rows,
             waves_r(f.c.kind) * f.c.tiles_r, (int)a->vocab, 1, (float)a->smoothing}, s);
  if (reduced)
    hipLaunchKernelGGL(k_loss_sum, 1, 1024, 0, s, (const float*)each, a->target, a->ignore_index, (int)a->rows,
                       (int)(a->reduction == FO_LOSS_MEAN), a->loss, a->count);
  return launch_check("loss forward launch");
}

// What lse's rounding left, from the forward pass's statistics made again: the same tiles
// of the same sums (pieces are whole tiles), so the same bits.
template <typename T>
const float* find_rest(const fo_loss* a, const LossBackward& b, const Operand& x, Packing& pack, hipStream_t s) {
  const int64_t es = elem_bytes<T>;
  v2f* part = (v2f*)at(a->workspace, b.part);
  float* rest = (float*)at(a->workspace, b.rest);
  for (int64_t first = 0; first < a->vocab; first += b.piece) {
    const int64_t nv = std::min(b.piece, a->vocab - first), tile = tile_r(b.statistics.kind);
    const Operand w = pack.operand(static_cast<const uint8_t*>(a->weight) + first * a->weight_ld * es, a->weight_ld, nv,
                                   a->cols, b.w, b.k);
    pack.launch(s);
    Cut c = b.statistics;
    c.tiles_r = (int)((nv + tile - 1) / tile);
    launch_product<T, Statistics, ROWS_ROWS>(
        product_of(w, nv, x, a->rows, b.k, es), c,
        {part + first / tile * waves_r(c.kind) * a->rows, nullptr, nullptr, a->target, a->ignore_index}, s);
  }
  join_rows({part, nullptr, nullptr, a->target, nullptr, nullptr, a->lse, rest, a->ignore_index, (int)a->rows, (int)b.parts,
             (int)a->vocab, 1, 0.0f}, s);
  return rest;
}

template <typename T>
int run_loss_backward(const fo_loss* a, const float* rest, const LossBackward& b, hipStream_t s) {
  const int64_t es = elem_bytes<T>;
  void* ws = a->workspace;
  // a token's gradient is a common factor times its unit: 1 with a reduction
  float *unit = (float*)at(ws, b.unit), *largest = (float*)at(ws, b.factor);
  Factor factor = {a->dloss, a->reduction == FO_LOSS_MEAN ? a->count : nullptr};
  if (unit) {
    hipLaunchKernelGGL(k_loss_factors, 1, 1024, 0, s, a->dloss, a->dloss_ld, a->target, a->ignore_index, (int)a->rows, unit,
                       largest);
    factor = {largest, nullptr};
  }
  Packing pack = {a->dtype, ws};
  const Operand x = pack.operand(a->x, a->x_ld, a->rows, a->cols, b.x, b.k);
  // dweight reads x without the tokens that are not counted: 0 times what they hold need not be 0
  Operand xm = {};
  if (a->dweight) xm = pack.copy(a->x, a->x_ld, a->rows, a->cols, b.xm, b.k, b.n, a->target, a->ignore_index);
  if (!rest) rest = find_rest<T>(a, b, x, pack, s);
  // half precision holds gradients of logits times 2^15
  const float scale = __is_same(T, Fp16) ? 32768.0f : 1.0f;
  const int64_t slice = a->rows * b.sums_ld;
  for (int64_t first = 0; first < a->vocab; first += b.piece) {
    const int64_t nv = std::min(b.piece, a->vocab - first), nvp = padded(nv);
    const Operand w = pack.operand(static_cast<const uint8_t*>(a->weight) + first * a->weight_ld * es, a->weight_ld, nv,
                                   a->cols, b.w, b.k);
    pack.launch(s);
    const Operand dz = {at(ws, b.dz), nvp + kGap};
    const Product pz = product_of(w, nv, x, a->rows, b.k, es);
    // tokens in whole steps: the padding is written too (as zeros)
    launch_product<T, LogitGradients, ROWS_ROWS>(
        pz, b.logits(nv, a->rows),
        {at(ws, b.dz), dz.ld, a->lse, rest, unit, a->target, a->ignore_index, (int)first, (int)a->vocab, (int)b.n, scale,
         (float)a->smoothing}, s);
    if (a->dx) {
      Product px = product_of(w, a->cols, dz, a->rows, nvp, es);
      px.k = (int)nv;
      if (b.sums >= 0)
        launch_product<T, KeepSums, COLS_ROWS>(px, b.dx, {(float*)at(ws, b.sums), b.sums_ld, slice, first > 0}, s);
      else
        launch_product<T, StoreScaled, COLS_ROWS>(
            px, b.dx, {a->dx, nullptr, (int)a->rows, (int)a->rows, 0, a->cols, factor, 1.0f / scale, a->target, a->ignore_index}, s);
    }
    if (a->dweight) {
      const Product pw = product_of(xm, a->cols, dz, nv, b.n, es);
      launch_product<T, StoreScaled, COLS_COLS>(
          pw, cut(a->dtype, a->cols, nv, pw.steps, false, true, false),
          {static_cast<uint8_t*>(a->dweight) + first * a->cols * es, nullptr, (int)nv, (int)nv, 0, a->cols, factor,
           1.0f / scale, nullptr, 0}, s);
    }
  }
  if (a->dx && b.sums >= 0) {
    const JoinArgs j = {(const float*)at(ws, b.sums), b.sums_ld, slice, b.dx.slices, a->dx, factor, a->target,
                        a->ignore_index, (int)a->rows, (int)a->cols, 1.0f / scale};
    hipLaunchKernelGGL((k_join<T>), grid_of((slice / 4 + 255) / 256), 256, 0, s, j);
  }
  return launch_check("loss backward launch");
}

// ---------------------------------------------------------------------------
// the gated block
// ---------------------------------------------------------------------------
int gated_checks(const fo_gated* a) {
  if (!a) return fail(FO_EINVAL, "args is NULL");
  if (!dtype_ok(a->dtype)) return fail(FO_EINVAL, "bad element type %d", a->dtype);
  if (a->activation < FO_SILU || a->activation > FO_GELU_TANH) return fail(FO_EINVAL, "bad activation %d", a->activation);
  if (a->rows < 0 || a->rows > kMaxTokens) return fail(FO_EINVAL, "rows = %lld is not in [0, 2^21]", (long long)a->rows);
  if (a->cols < 1 || a->cols > kMaxCols) return fail(FO_EINVAL, "cols = %lld is not in [1, 2^20]", (long long)a->cols);
  if (a->features < 1 || a->features > kMaxFeatures)
    return fail(FO_EINVAL, "features = %lld is not in [1, 2^20]", (long long)a->features);
  FO_TRY(area_check(a->rows, a->cols, 2 * a->features));
  if (!a->g != !a->u) return fail(FO_EINVAL, "g and u go together");
  return FO_OK;
}

int gated_inputs(const fo_gated* a, Arrays& ar, bool backward) {
  const size_t es = elem_size(a->dtype);
  const bool any = a->rows > 0;
  FO_TRY(ar.add(a->x, "x", false, any, a->rows, a->cols, a->x_ld, es));
  FO_TRY(ar.add(a->gate, "gate", false, any, a->features, a->cols, a->gate_ld, es));
  FO_TRY(ar.add(a->up, "up", false, any, a->features, a->cols, a->up_ld, es));
  FO_TRY(ar.add(a->g, "g", !backward, any && backward, a->rows, a->features, a->features, 4));
  FO_TRY(ar.add(a->u, "u", !backward, any && backward, a->rows, a->features, a->features, 4));
  return FO_OK;
}

template <typename T>
int run_gated_forward(const fo_gated* a, const GatedForward& f, hipStream_t s) {
  const int64_t es = elem_bytes<T>;
  Packing pack = {a->dtype, a->workspace};
  const Operand x = pack.operand(a->x, a->x_ld, a->rows, a->cols, f.x, f.k);
  const Operand gate = pack.operand(a->gate, a->gate_ld, a->features, a->cols, f.gate, f.k);
  const Operand up_w = pack.operand(a->up, a->up_ld, a->features, a->cols, f.up, f.k);
  pack.launch(s);
  Product p = product_of(gate, a->features, x, a->rows, f.k, es);
  p.r2 = up_w.p;
  launch_product<T, Gated, DUAL_ROWS>(p, f.c, {a->y, a->g, a->u, a->activation}, s);
  return launch_check("gated forward launch");
}

template <typename T>
int run_gated_backward(const fo_gated* a, const GatedBackward& b, hipStream_t s) {
  const int64_t es = elem_bytes<T>, half = b.half;
  void* ws = a->workspace;
  const GatedBwd g = {a->dy, a->dy_ld, a->g, a->u, at(ws, b.d), (int)a->rows, (int)b.n, (int)a->features, (int)half,
                      2 * half + kGap, a->activation};
  hipLaunchKernelGGL((k_gated_bwd<T>), grid_of((b.n * half / 8 + 255) / 256), 256, 0, s, g);
  const Operand d = {at(ws, b.d), g.ld};
  Packing pack = {a->dtype, ws};
  const Operand gate = pack.operand(a->gate, a->gate_ld, a->features, a->cols, b.gate, b.k);
  const Operand up_w = pack.operand(a->up, a->up_ld, a->features, a->cols, b.up, b.k);
  const Operand x = pack.operand(a->x, a->x_ld, a->rows, a->cols, b.x, b.k);
  pack.launch(s);
  if (a->dx) {
    Product p = product_of(gate, a->cols, d, a->rows, 2 * half, es);
    p.r2 = up_w.p;
    p.k = (int)a->features;
    p.joint = (int)(half * es / 128);
    if (b.dx.slices > 1) {
      const int64_t slice = a->rows * b.sums_ld;
      launch_product<T, KeepSums, COLS_ROWS>(p, b.dx, {(float*)at(ws, b.sums), b.sums_ld, slice, 0}, s);
      const JoinArgs j = {(const float*)at(ws, b.sums), b.sums_ld, slice, b.dx.slices, a->dx, {nullptr, nullptr}, nullptr, 0,
                          (int)a->rows, (int)a->cols, 1.0f};
      hipLaunchKernelGGL((k_join<T>), grid_of((slice / 4 + 255) / 256), 256, 0, s, j);
    } else {
      launch_product<T, StoreScaled, COLS_ROWS>(p, b.dx, {a->dx, nullptr, (int)a->rows, (int)a->rows, 0, a->cols, {nullptr, nullptr}, 1.0f, nullptr, 0}, s);
    }
  }
  if (a->dgate || a->dup) {
    Product p = product_of(x, a->cols, d, 2 * half, b.n, es);
    p.k = (int)a->rows;
    launch_product<T, StoreScaled, COLS_COLS>(
        p, cut(a->dtype, a->cols, 2 * half, p.steps, false, true, false),
        {a->dgate, a->dup, (int)half, (int)a->features, (int)a->features, a->cols, {nullptr, nullptr}, 1.0f, nullptr, 0}, s);
  }
  return launch_check("gated backward launch");
}

}  // namespace

extern "C" {

int fo_loss_forward_workspace(const fo_loss* a, int64_t* bytes) {
  clear_error();
  if (!bytes) return fail(FO_EINVAL, "bytes is NULL");
  FO_TRY(loss_checks(a));
  *bytes = a->rows ? loss_forward(a).bytes : 0;
  return FO_OK;
}

static int loss_forward_call(const fo_loss* a, float* rest, bool wanted, void* stream) {
  clear_error();
  FO_TRY(loss_checks(a));
  const bool any = a->rows > 0, reduced = a->reduction != FO_LOSS_NONE;
  Arrays ar;
  FO_TRY(loss_inputs(a, ar));
  FO_TRY(ar.add(a->loss, "loss", true, any || reduced, reduced ? 1 : a->rows, 1, 1, 4));
  FO_TRY(ar.add(a->lse, "lse", true, any, a->rows, 1, 1, 4));
  FO_TRY(ar.add(rest, "rest", true, wanted && any, a->rows, 1, 1, 4));
  FO_TRY(ar.add(a->count, "count", true, reduced, 1, 1, 1, 4));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!any) {
    FO_TRY(ar.disjoint());
    if (!reduced) return FO_OK;
    hipLaunchKernelGGL(k_loss_sum, 1, 1024, 0, s, (const float*)nullptr, a->target, a->ignore_index, 0,
                       (int)(a->reduction == FO_LOSS_MEAN), a->loss, a->count);
    return launch_check("loss forward launch");
  }
  const LossForward f = loss_forward(a);
  FO_TRY(workspace_check(a->workspace, a->workspace_bytes, f.bytes, ar));
  FO_TRY(ar.disjoint());
  if (a->dtype == FO_BF16) return run_loss_forward<Bf16>(a, rest, f, s);
  if (a->dtype == FO_FP16) return run_loss_forward<Fp16>(a, rest, f, s);
  return run_loss_forward<F32>(a, rest, f, s);
}
int fo_loss_forward(const fo_loss* a, void* stream) { return loss_forward_call(a, nullptr, false, stream); }
int fo_loss_forward_rest(const fo_loss* a, float* rest, void* stream) { return loss_forward_call(a, rest, true, stream); }

int fo_loss_backward_workspace(const fo_loss* a, int64_t* bytes) {
  clear_error();
  if (!bytes) return fail(FO_EINVAL, "bytes is NULL");
  FO_TRY(loss_checks(a));
  *bytes = a->rows ? loss_backward(a, a->dx, a->dweight).bytes : 0;
  return FO_OK;
}

static int loss_backward_call(const fo_loss* a, const float* rest, bool given, void* stream) {
  clear_error();
  FO_TRY(loss_checks(a));
  const size_t es = elem_size(a->dtype);
  const bool any = a->rows > 0, none = a->reduction == FO_LOSS_NONE;
  Arrays ar;
  FO_TRY(loss_inputs(a, ar));
  FO_TRY(ar.add(a->lse, "lse", false, any, a->rows, 1, 1, 4));
  FO_TRY(ar.add(rest, "rest", false, given && any, a->rows, 1, 1, 4));
  FO_TRY(ar.add(a->count, "count", false, a->reduction == FO_LOSS_MEAN && any, 1, 1, 1, 4));
  FO_TRY(ar.add(a->dloss, "dloss", false, any, none ? a->rows : 1, 1, none ? a->dloss_ld : 1, 4));
  FO_TRY(ar.add(a->dx, "dx", true, false, a->rows, a->cols, a->cols, es));
  FO_TRY(ar.add(a->dweight, "dweight", true, false, a->vocab, a->cols, a->cols, es));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((!a->dx || !any) && !a->dweight) return ar.disjoint();
  if (!any) {
    FO_TRY(ar.disjoint());
    const int64_t bytes = a->vocab * a->cols * (int64_t)es;
    hipLaunchKernelGGL(k_zero, grid_of((bytes + 4095) / 4096), 256, 0, s, a->dweight, bytes);
    return launch_check("loss backward launch");
  }
  const LossBackward b = loss_backward(a, a->dx, a->dweight);
  FO_TRY(workspace_check(a->workspace, a->workspace_bytes, b.bytes, ar));
  FO_TRY(ar.disjoint());
  if (a->dtype == FO_BF16) return run_loss_backward<Bf16>(a, rest, b, s);
  if (a->dtype == FO_FP16) return run_loss_backward<Fp16>(a, rest, b, s);
  return run_loss_backward<F32>(a, rest, b, s);
}
int fo_loss_backward(const fo_loss* a, void* stream) { return loss_backward_call(a, nullptr, false, stream); }
int fo_loss_backward_rest(const fo_loss* a, const float* rest, void* stream) { return loss_backward_call(a, rest, true, stream); }

int fo_gated_forward_workspace(const fo_gated* a, int64_t* bytes) {
  clear_error();
  if (!bytes) return fail(FO_EINVAL, "bytes is NULL");
  FO_TRY(gated_checks(a));
  *bytes = a->rows ? gated_forward(a).bytes : 0;
  return FO_OK;
}

int fo_gated_forward(const fo_gated* a, void* stream) {
  clear_error();
  FO_TRY(gated_checks(a));
  Arrays ar;
  FO_TRY(gated_inputs(a, ar, false));
  FO_TRY(ar.add(a->y, "y", true, a->rows > 0, a->rows, a->features, a->features, elem_size(a->dtype)));
  if (a->rows == 0) return ar.disjoint();
  const GatedForward f = gated_forward(a);
  FO_TRY(workspace_check(a->workspace, a->workspace_bytes, f.bytes, ar));
  FO_TRY(ar.disjoint());
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a->dtype == FO_BF16) return run_gated_forward<Bf16>(a, f, s);
  if (a->dtype == FO_FP16) return run_gated_forward<Fp16>(a, f, s);
  return run_gated_forward<F32>(a, f, s);
}

int fo_gated_backward_workspace(const fo_gated* a, int64_t* bytes) {
  clear_error();
  if (!bytes) return fail(FO_EINVAL, "bytes is NULL");
  FO_TRY(gated_checks(a));
  *bytes = a->rows ? gated_backward(a, a->dx, a->dgate || a->dup).bytes : 0;
  return FO_OK;
}

int fo_gated_backward(const fo_gated* a, void* stream) {
  clear_error();
  FO_TRY(gated_checks(a));
  const size_t es = elem_size(a->dtype);
  Arrays ar;
  FO_TRY(gated_inputs(a, ar, true));
  FO_TRY(ar.add(a->dy, "dy", false, a->rows > 0, a->rows, a->features, a->dy_ld, es));
  FO_TRY(ar.add(a->dx, "dx", true, false, a->rows, a->cols, a->cols, es));
  FO_TRY(ar.add(a->dgate, "dgate", true, false, a->features, a->cols, a->cols, es));
  FO_TRY(ar.add(a->dup, "dup", true, false, a->features, a->cols, a->cols, es));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((!a->dx || a->rows == 0) && !a->dgate && !a->dup) return ar.disjoint();
  if (a->rows == 0) {
    FO_TRY(ar.disjoint());
    const int64_t bytes = a->features * a->cols * (int64_t)es;
    for (void* out : {a->dgate, a->dup})
      if (out) hipLaunchKernelGGL(k_zero, grid_of((bytes + 4095) / 4096), 256, 0, s, out, bytes);
    return launch_check("gated backward launch");
  }
  const GatedBackward b = gated_backward(a, a->dx, a->dgate || a->dup);
  FO_TRY(workspace_check(a->workspace, a->workspace_bytes, b.bytes, ar));
  FO_TRY(ar.disjoint());
  if (a->dtype == FO_BF16) return run_gated_backward<Bf16>(a, b, s);
  if (a->dtype == FO_FP16) return run_gated_backward<Fp16>(a, b, s);
  return run_gated_backward<F32>(a, b, s);
}

}  // extern "C"
