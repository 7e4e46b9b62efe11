// fo_products_args.hpp -- host-only half of the products' launcher: limits, how a
// product is cut into tiles and slices, and where a workspace's parts lie.  No HIP:
// tests/host/products_args_check.cpp compiles it alone.
#pragma once

#include <stdint.h>
#include <stddef.h>

#include <algorithm>

#include "../../include/foamd.h"
#include "fo_error.hpp"
#include "fo_rows_args.hpp"

namespace fo {
namespace prod {

using rows::dtype_ok;
using rows::elem_size;

// A tile's rows are addressed by 32-bit offsets: 256 rows of at most 2^23 bytes.
constexpr int64_t kMaxRowBytes = int64_t(1) << 23;
constexpr int64_t kMaxTokens = int64_t(1) << 21, kMaxCols = int64_t(1) << 20, kMaxFeatures = int64_t(1) << 20;
constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr int64_t kMaxLogits = int64_t(1) << 38;      // tokens * vocab: a launch's threads fit 32 bits

inline int64_t up(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }
inline int64_t padded(int64_t n) { return up(n, 64); }          // whole steps of every type

// Whether rows can be read as they lie: whole steps, 16-byte aligned.
inline bool direct(const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype) {
  const int64_t es = (int64_t)elem_size(dtype), step = 128 / es;
  if (reinterpret_cast<uintptr_t>(p) % 16 || cols % step) return false;
  return rows == 1 || (ld * es % 16 == 0 && ld * es <= kMaxRowBytes);
}

// Parts of a workspace, one after another.
struct Layout {
  int64_t bytes = 0;
  int64_t take(int64_t n) {
    const int64_t at = bytes;
    bytes += up(n, 256);
    return at;
  }
};

// Tile kinds of k_product (R x C).
enum TileKind { WIDE, MIDDLE, SMALL, NARROW };
struct Cut { TileKind kind; int tiles_r, tiles_c, slices; };
constexpr int tile_r(TileKind k) { return k == WIDE ? 256 : k == MIDDLE ? 128 : 64; }
constexpr int tile_c(TileKind k) { return k == WIDE ? 256 : k == MIDDLE ? 128 : k == SMALL ? 64 : 32; }
// waves that share a tile's rows of R: each has a part of them to itself
constexpr int waves_r(TileKind k) { return k == WIDE || k == MIDDLE ? 2 : 1; }
constexpr int64_t kUnits = 256;                                 // compute units

// nr (with `dual`, of each of two matrices) rows of R against nc of C, `steps` of k.
inline Cut cut(int64_t nr, int64_t nc, int64_t steps, bool dual, bool narrow_ok, bool sliced) {
  const int64_t all_r = dual ? 2 * up(nr, 32) : nr;
  Cut c = {};
  auto tiles = [&](TileKind k) {
    c.kind = k;
    c.tiles_r = (int)((all_r + tile_r(k) - 1) / tile_r(k));
    c.tiles_c = (int)((nc + tile_c(k) - 1) / tile_c(k));
    return (int64_t)c.tiles_r * c.tiles_c;
  };
  int64_t n;
  if (narrow_ok && nc <= 32) n = tiles(NARROW);
  else if ((n = tiles(WIDE)) < kUnits && (n = tiles(MIDDLE)) < kUnits) n = tiles(SMALL);
  c.slices = 1;
  if (sliced) c.slices = (int)std::max<int64_t>(1, std::min<int64_t>({2 * kUnits / n, steps / 8, 32}));
  return c;
}

// Vocabulary per piece of the backward pass: the logits' gradients of a piece are at
// most about 2^28 elements (512 MB in 16 bits).
constexpr int64_t kPieceElems = int64_t(1) << 28;
inline int64_t piece_vocab(int64_t tokens, int64_t vocab) {
  const int64_t most = std::max<int64_t>(1024, kPieceElems / padded(tokens));
  const int64_t pieces = (vocab + most - 1) / most;
  return std::min(up((vocab + pieces - 1) / pieces, 256), padded(vocab));
}

// What a loss call's workspace holds (offsets; -1: not there).
struct LossForward {
  int64_t x = -1, w = -1, part = 0, sums = -1, chosen = 0, each = -1, bytes = 0;
  int64_t k = 0;                                                // columns, whole steps
  Cut c = {};
};
inline LossForward loss_forward(const fo_loss* a) {
  LossForward f;
  Layout l;
  const int64_t es = (int64_t)elem_size(a->dtype);
  f.k = a->cols % (128 / es) ? padded(a->cols) : a->cols;
  if (!direct(a->x, a->rows, a->cols, a->x_ld, a->dtype)) f.x = l.take(a->rows * f.k * es);
  if (!direct(a->weight, a->vocab, a->cols, a->weight_ld, a->dtype)) f.w = l.take(a->vocab * f.k * es);
  f.c = cut(a->vocab, a->rows, f.k * es / 128, false, true, false);
  const int64_t parts = (int64_t)waves_r(f.c.kind) * f.c.tiles_r;
  f.part = l.take(parts * a->rows * 8);
  if (a->smoothing != 0.0) f.sums = l.take(parts * a->rows * 4);
  f.chosen = l.take(a->rows * 4);
  if (a->reduction != FO_LOSS_NONE) f.each = l.take(a->rows * 4);
  f.bytes = l.bytes;
  return f;
}

struct LossBackward {
  int64_t unit, factor, x = -1, w = -1, xm = -1, dz = -1, sums = -1, bytes = 0;
  int64_t k, n, piece, sums_ld;                                 // columns and tokens in whole steps; vocabulary per piece
  Cut dx = {};                                                  // of a whole piece
};
inline LossBackward loss_backward(const fo_loss* a, bool dx, bool dw) {
  LossBackward b;
  Layout l;
  const int64_t es = (int64_t)elem_size(a->dtype);
  b.k = a->cols % (128 / es) ? padded(a->cols) : a->cols;
  b.n = padded(a->rows);
  b.piece = piece_vocab(a->rows, a->vocab);
  b.unit = l.take(a->rows * 4);
  b.factor = l.take(4);
  if (!direct(a->x, a->rows, a->cols, a->x_ld, a->dtype)) b.x = l.take(a->rows * b.k * es);
  if (!direct(a->weight, a->vocab, a->cols, a->weight_ld, a->dtype)) b.w = l.take(std::min(b.piece, a->vocab) * b.k * es);
  if (dw) b.xm = l.take(b.n * b.k * es);
  b.dz = l.take(b.n * b.piece * es);
  b.sums_ld = up(a->cols, 4);
  if (dx) {
    b.dx = cut(a->cols, a->rows, b.piece * es / 128, false, true, true);
    b.sums = l.take((int64_t)b.dx.slices * a->rows * b.sums_ld * 4);
  }
  b.bytes = l.bytes;
  return b;
}

struct GatedForward { int64_t x = -1, gate = -1, up = -1, bytes = 0, k = 0; Cut c = {}; };
inline GatedForward gated_forward(const fo_gated* a) {
  GatedForward f;
  Layout l;
  const int64_t es = (int64_t)elem_size(a->dtype);
  f.k = a->cols % (128 / es) ? padded(a->cols) : a->cols;
  if (!direct(a->x, a->rows, a->cols, a->x_ld, a->dtype)) f.x = l.take(a->rows * f.k * es);
  // both weights are read with one row stride
  if (!direct(a->gate, a->features, a->cols, a->gate_ld, a->dtype) ||
      !direct(a->up, a->features, a->cols, a->up_ld, a->dtype) || a->gate_ld != a->up_ld) {
    f.gate = l.take(a->features * f.k * es);
    f.up = l.take(a->features * f.k * es);
  }
  f.c = cut(a->features, a->rows, f.k * es / 128, true, true, false);
  f.bytes = l.bytes;
  return f;
}

struct GatedBackward {
  int64_t d = -1, x = -1, gate = -1, up = -1, sums = -1, bytes = 0;
  int64_t k, half, n, sums_ld;
  Cut dx = {};
};
inline GatedBackward gated_backward(const fo_gated* a, bool dx, bool dw) {
  GatedBackward b;
  Layout l;
  const int64_t es = (int64_t)elem_size(a->dtype);
  b.k = a->cols % (128 / es) ? padded(a->cols) : a->cols;
  b.half = padded(a->features);
  b.n = padded(a->rows);
  b.sums_ld = up(a->cols, 4);
  b.d = l.take(b.n * 2 * b.half * es);
  if (dx) {
    if (!direct(a->gate, a->features, a->cols, a->gate_ld, a->dtype) ||
        !direct(a->up, a->features, a->cols, a->up_ld, a->dtype) || a->gate_ld != a->up_ld) {
      b.gate = l.take(a->features * b.k * es);
      b.up = l.take(a->features * b.k * es);
    }
    b.dx = cut(a->cols, a->rows, 2 * b.half * es / 128, false, true, true);
    if (b.dx.slices > 1) b.sums = l.take((int64_t)b.dx.slices * a->rows * b.sums_ld * 4);
  }
  if (dw && !direct(a->x, a->rows, a->cols, a->x_ld, a->dtype)) b.x = l.take(a->rows * b.k * es);
  b.bytes = l.bytes;
  return b;
}

}  // namespace prod
}  // namespace fo
