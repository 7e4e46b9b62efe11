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

// A tile's rows are addressed by 32-bit offsets: 256 rows of at most 2^23 bytes (and a gap).
constexpr int64_t kMaxRowBytes = int64_t(1) << 23;
constexpr int64_t kMaxTokens = int64_t(1) << 21, kMaxCols = int64_t(1) << 20, kMaxFeatures = int64_t(1) << 20;
constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr int64_t kMaxArea = int64_t(1) << 36;        // of any two of a product's sizes: a launch's threads fit 32 bits

inline int64_t up(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }
inline int64_t padded(int64_t n) { return up(n, 64); }          // whole steps of every type

// Whether rows can be read as they lie: whole steps, 16-byte aligned.
inline bool direct(const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype) {
  const int64_t es = (int64_t)elem_size(dtype), step = 128 / es;
  if (reinterpret_cast<uintptr_t>(p) % 16 || cols % step) return false;
  return rows == 1 || (ld * es % 16 == 0 && ld * es <= kMaxRowBytes);
}

// Elements between rows of gradients in a workspace.  Rows 64 KB apart, which the sizes of
// models give (32768 places in 16 bits), send a tile's 256 rows to the same few memory
// channels: 8192 x 768 x 32768 took 486 us, with the gap 395 us.
constexpr int64_t kGap = 64;

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
// of a workgroup (a small tile's are two groups of waves)
constexpr int threads(TileKind k) { return k == WIDE ? 512 : k == NARROW ? 64 : 256; }
constexpr int64_t kUnits = 256;                                 // compute units

// What a product takes, in microseconds, by the times measured on the card (`steps` of
// one round: all compute units once).  A round of wide tiles is 256 of them, one per
// compute unit, of the others 512; a last round of half of that or less takes the second
// figure of each pair.  16-bit types: 1.67 per step (wide), 0.94 and 0.59 (middle), 0.36
// and 0.31 (small); float32, whose matrix instructions take 8 times as long, 7.4, 4 and
// 2, 1.1 and 0.6.  What a
// round takes besides its steps differs with the epilogue (4 to 15, 2 to 8 and 3 to 5):
// its middle is taken.  (Since these were measured the main loop has become 3 to 5 %
// faster, wide and middle tiles alike.)
inline double round_time(TileKind k, bool f32, bool half, double steps) {
  const double fixed = k == WIDE ? 9.0 : k == MIDDLE ? 4.5 : 4.0;
  const double step = f32 ? (k == WIDE ? 7.4 : k == MIDDLE ? (half ? 2.0 : 4.0) : (half ? 0.6 : 1.1))
                          : (k == WIDE ? 1.67 : k == MIDDLE ? (half ? 0.59 : 0.94) : (half ? 0.31 : 0.36));
  return fixed + step * steps;
}
inline double product_time(TileKind k, bool f32, int64_t tiles, int64_t slices, int64_t steps) {
  const int64_t slots = k == WIDE ? kUnits : 2 * kUnits, n = tiles * slices, last = n % slots;
  const double each = (double)((steps + slices - 1) / slices);
  return (double)(n / slots) * round_time(k, f32, false, each) +
         (last ? round_time(k, f32, k != WIDE && last <= kUnits, each) : 0.0);
}

inline Cut tiles_of(TileKind k, int64_t nr, int64_t nc) {
  return {k, (int)((nr + tile_r(k) - 1) / tile_r(k)), (int)((nc + tile_c(k) - 1) / tile_c(k)), 1};
}

// How nr (with `dual`, of each of two matrices) rows of R against nc of C, `steps` of k,
// are cut: the kind of tile, and with `sliced` the number of slices of k (whose sums are
// written and read once more, 4 bytes each way at 5 TB/s), that take the least time.
// Up to 32 rows of C go in narrow tiles, which waste least on rows that are not there.
inline Cut cut(int dtype, int64_t nr, int64_t nc, int64_t steps, bool dual, bool narrow_ok, bool sliced) {
  const int64_t all_r = dual ? 2 * up(nr, 32) : nr;
  const bool f32 = dtype == FO_F32;
  auto tiles = [&](TileKind k) { return tiles_of(k, all_r, nc); };
  // at most 32, and 1 GB of sums
  const int64_t most = sliced ? std::max<int64_t>(1, std::min<int64_t>(32, (int64_t(1) << 28) / (nr * nc))) : 1;
  auto slices = [&](Cut c) {
    const int64_t n = (int64_t)c.tiles_r * c.tiles_c;
    return (int)std::max<int64_t>(1, std::min<int64_t>({2 * kUnits / n, steps / 8, most}));
  };
  if (narrow_ok && nc <= 32) {
    Cut c = tiles(NARROW);
    if (sliced) c.slices = slices(c);
    return c;
  }
  Cut best = {};
  double least = 0.0;
  for (TileKind k : {WIDE, MIDDLE, SMALL}) {
    Cut c = tiles(k);
    const int64_t n = (int64_t)c.tiles_r * c.tiles_c;
    // float32 sums of long k are also cut for their accuracy: chains of at most 2048 terms.
    // Where slices cannot see to that, wide tiles, whose sums are one chain, are not taken:
    // 32768 equal terms are off by up to 4.9e-4 in them, 9e-6 in the others' two levels.
    // 8192 x 4096 x 14336 takes 13.17 ms forward against 12.82, its gradients 28.4 against
    // 27.6; 4096 x 4096 x 32000 of a loss 7.55 against 7.33 and 23.2 against 22.7.
    const int fewest = f32 ? (int)std::min((steps + 63) / 64, most) : 1;
    for (int s = fewest; s <= most && (s == fewest || steps / s >= 8); ++s) {
      if (f32 && k == WIDE && (steps + s - 1) / s > 64) continue;
      const double t = product_time(k, f32, n, s, steps) + (sliced ? (double)s * (double)nr * (double)nc * 8e-6 / 5.0 : 0.0);
      if (best.slices && t >= least) continue;
      best = c;
      best.slices = s;
      least = t;
    }
  }
  return best;
}
// (the time that cut() expects)
inline double cut_time(int dtype, const Cut& c, int64_t steps) {
  return c.kind == NARROW ? 0.0
                          : product_time(c.kind, dtype == FO_F32, (int64_t)c.tiles_r * c.tiles_c, c.slices, steps);
}

// Vocabulary per piece of the backward pass: the logits' gradients of a piece are at
// most 2^28 elements (512 MB in 16 bits), and a little padding, or 1024 places of every
// token where that is more (past 2^18 tokens).  Of the sizes down to half of that the
// one whose three products fill the card's last rounds best (8192 tokens, 768 columns,
// 50257 places: 21504 instead of 25344, whose weight gradients are 297 wide tiles on 256
// compute units).  Where there are several they are multiples of 256: whole tiles of any kind.
constexpr int64_t kPieceElems = int64_t(1) << 28;
// (`kind`: of the tiles that make the logits)
inline int64_t piece_vocab(int dtype, int64_t tokens, int64_t cols, int64_t vocab, TileKind kind) {
  const int64_t es = (int64_t)elem_size(dtype), n = padded(tokens);
  const int64_t most = std::min(std::max<int64_t>(1024, kPieceElems / n / 256 * 256), kMaxRowBytes / 4);
  if (vocab <= most) return padded(vocab);
  const int64_t steps_d = (cols * es + 127) / 128, steps_n = n * es / 128;
  auto time = [&](int64_t nv) {
    const int64_t steps_v = padded(nv) * es / 128;
    return cut_time(dtype, tiles_of(kind, nv, n), steps_d) +
           cut_time(dtype, cut(dtype, cols, tokens, steps_v, false, true, true), steps_v) +
           cut_time(dtype, cut(dtype, cols, nv, steps_n, false, true, false), steps_n);
  };
  int64_t best = most;
  double least = 0.0;
  for (int64_t nv = most; 2 * nv >= most && nv >= 1024; nv -= std::max<int64_t>(256, most / 16 / 256 * 256)) {
    const double t = (double)(vocab / nv) * time(nv) + (vocab % nv ? time(vocab % nv) : 0.0);
    if (nv != most && t >= least) continue;
    best = nv;
    least = t;
  }
  return best;
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
  f.c = cut(a->dtype, a->vocab, a->rows, f.k * es / 128, false, true, false);
  const int64_t parts = (int64_t)waves_r(f.c.kind) * f.c.tiles_r;
  f.part = l.take(parts * a->rows * 8);
  if (a->smoothing != 0.0) f.sums = l.take(parts * a->rows * 4);
  f.chosen = l.take(a->rows * 4);
  if (a->reduction != FO_LOSS_NONE) f.each = l.take(a->rows * 4);
  f.bytes = l.bytes;
  return f;
}

struct LossBackward {
  int64_t unit = -1, factor = -1, rest = -1, x = -1, w = -1, xm = -1, dz = -1, sums = -1, bytes = 0;
  // The forward pass's tiles.  The logits are made again in tiles of the same kind, whose sums
  // add up in the same order: the same bits, so that what they are off by cancels in exp(z - lse).
  // (With tiles chosen for themselves, small ones for the narrow tiles of 32 tokens and fewer, float32
  // gradients of 22 x 386 x 13 were off by 7e-6 instead of 6e-7, and probabilities added up to 1 only
  // as well as two ways of adding a logit agree.)
  Cut statistics = {};
  // without the forward pass's `rest`: its statistics again, where dz comes later
  int64_t part = -1, parts = 0;
  // tiles of a piece of nv places: all tokens of whole steps, or of a narrow tile
  Cut logits(int64_t nv, int64_t rows) const {
    return tiles_of(statistics.kind, nv, statistics.kind == NARROW ? rows : n);
  }
  int64_t k, n, piece, sums_ld;                                 // columns and tokens in whole steps; vocabulary per piece
  Cut dx = {};                                                  // of a whole piece
};
inline LossBackward loss_backward(const fo_loss* a, bool dx, bool dw) {
  LossBackward b;
  Layout l;
  const int64_t es = (int64_t)elem_size(a->dtype);
  b.k = a->cols % (128 / es) ? padded(a->cols) : a->cols;
  b.n = padded(a->rows);
  b.statistics = cut(a->dtype, a->vocab, a->rows, b.k * es / 128, false, true, false);
  b.piece = piece_vocab(a->dtype, a->rows, a->cols, a->vocab, b.statistics.kind);
  if (a->reduction == FO_LOSS_NONE) {
    b.unit = l.take(a->rows * 4);
    b.factor = l.take(4);
  }
  if (!direct(a->x, a->rows, a->cols, a->x_ld, a->dtype)) b.x = l.take(a->rows * b.k * es);
  if (!direct(a->weight, a->vocab, a->cols, a->weight_ld, a->dtype)) b.w = l.take(std::min(b.piece, a->vocab) * b.k * es);
  if (dw) b.xm = l.take(b.n * b.k * es);
  b.rest = l.take(a->rows * 4);
  b.parts = (int64_t)waves_r(b.statistics.kind) * b.statistics.tiles_r;
  b.part = b.dz = l.take(std::max(b.n * (b.piece + kGap) * es, b.parts * a->rows * 8));
  b.sums_ld = up(a->cols, 4);
  if (dx) {
    b.dx = cut(a->dtype, a->cols, a->rows, b.piece * es / 128, false, true, true);
    if (b.dx.slices > 1 || a->vocab > b.piece) b.sums = l.take((int64_t)b.dx.slices * a->rows * b.sums_ld * 4);
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
  f.c = cut(a->dtype, a->features, a->rows, f.k * es / 128, true, true, false);
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
  b.d = l.take(b.n * (2 * b.half + kGap) * es);
  if (dx) {
    if (!direct(a->gate, a->features, a->cols, a->gate_ld, a->dtype) ||
        !direct(a->up, a->features, a->cols, a->up_ld, a->dtype) || a->gate_ld != a->up_ld) {
      b.gate = l.take(a->features * b.k * es);
      b.up = l.take(a->features * b.k * es);
    }
    b.dx = cut(a->dtype, a->cols, a->rows, 2 * b.half * es / 128, false, true, true);
    if (b.dx.slices > 1) b.sums = l.take((int64_t)b.dx.slices * a->rows * b.sums_ld * 4);
  }
  if (dw && !direct(a->x, a->rows, a->cols, a->x_ld, a->dtype)) b.x = l.take(a->rows * b.k * es);
  b.bytes = l.bytes;
  return b;
}

}  // namespace prod
}  // namespace fo
