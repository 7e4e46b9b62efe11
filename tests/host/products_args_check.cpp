// The host half of the products' launcher (csrc/fo_products_args.hpp) against brute
// force: tiles cover their rows, slices have steps, pieces cover the vocabulary within
// the 32-bit offsets of a tile, launches fit their limits, and a workspace's parts
// neither overlap nor pass its size.
#include <cstdarg>
#include <cstdio>
#include <random>
#include <vector>

#include "../../precision_optimizer_state_amd/csrc/fo_products_args.hpp"

int fo::fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return code;
}
void fo::clear_error() {}

using namespace fo::prod;

#define CHECK(c)                                                     \
  do {                                                               \
    if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return false; } \
  } while (0)

static bool covers(const Cut& c, int64_t nr, int64_t nc, int64_t steps, bool dual) {
  const int64_t all_r = dual ? 2 * up(nr, 32) : nr;
  CHECK(c.tiles_r >= 1 && c.tiles_c >= 1 && c.slices >= 1 && c.slices <= 32);
  CHECK((int64_t)c.tiles_r * tile_r(c.kind) >= all_r && (int64_t)(c.tiles_r - 1) * tile_r(c.kind) < all_r);
  CHECK((int64_t)c.tiles_c * tile_c(c.kind) >= nc && (int64_t)(c.tiles_c - 1) * tile_c(c.kind) < nc);
  CHECK(c.slices == 1 || steps >= c.slices);
  // tiles, workgroups and threads of a launch are 32-bit
  const int64_t threads = c.kind == WIDE ? 512 : c.kind == MIDDLE ? 256 : c.kind == SMALL ? 128 : 64;
  CHECK((__int128)c.tiles_r * c.tiles_c * c.slices * threads < ((__int128)1 << 32));
  return true;
}

struct Part { int64_t at, bytes; };
static bool apart(std::vector<Part> parts, int64_t total) {
  for (size_t i = 0; i < parts.size(); ++i) {
    if (parts[i].at < 0) continue;
    CHECK(parts[i].at % 256 == 0 && parts[i].at + parts[i].bytes <= total);
    for (size_t j = 0; j < i; ++j)
      CHECK(parts[j].at < 0 || parts[i].at >= parts[j].at + parts[j].bytes || parts[j].at >= parts[i].at + parts[i].bytes);
  }
  return true;
}

static bool loss(const fo_loss& a) {
  const int64_t es = (int64_t)elem_size(a.dtype);
  const LossForward f = loss_forward(&a);
  CHECK(f.k >= a.cols && f.k * es % 128 == 0);
  CHECK(f.x < 0 ? direct(a.x, a.rows, a.cols, a.x_ld, a.dtype) : true);
  CHECK(covers(f.c, a.vocab, a.rows, f.k * es / 128, false));
  const int64_t parts = (int64_t)waves_r(f.c.kind) * f.c.tiles_r;
  CHECK(apart({{f.x, a.rows * f.k * es}, {f.w, a.vocab * f.k * es}, {f.part, parts * a.rows * 8}, {f.sums, parts * a.rows * 4},
               {f.chosen, a.rows * 4}, {f.each, a.rows * 4}}, f.bytes));
  for (int need = 1; need < 4; ++need) {
    const bool dx = need & 1, dw = need & 2;
    const LossBackward b = loss_backward(&a, dx, dw);
    CHECK(b.n % 64 == 0 && b.n >= a.rows && b.n - a.rows < 64 && b.n * b.k <= ((int64_t)1 << 62));
    CHECK(b.piece % 64 == 0 && b.piece * es <= kMaxRowBytes && b.piece >= std::min<int64_t>(a.vocab, 1024));
    CHECK(b.n * b.piece <= 2 * kPieceElems || b.piece <= 1024);
    for (int64_t nv : {std::min(b.piece, a.vocab), a.vocab % b.piece ? a.vocab % b.piece : std::min(b.piece, a.vocab)}) {
      CHECK(covers(cut(a.dtype, nv, b.n, b.k * es / 128, false, false, false), nv, b.n, b.k * es / 128, false));
      CHECK(covers(cut(a.dtype, a.cols, nv, b.n * es / 128, false, true, false), a.cols, nv, b.n * es / 128, false));
      // gradients of logits are written in whole tiles of at least 64 rows of C: b.n of them
      CHECK(tile_c(cut(a.dtype, nv, b.n, b.k * es / 128, false, false, false).kind) >= 64);
    }
    if (dx) CHECK(covers(b.dx, a.cols, a.rows, b.piece * es / 128, false));
    CHECK(apart({{b.unit, a.rows * 4}, {b.factor, 4}, {b.x, a.rows * b.k * es}, {b.w, std::min(b.piece, a.vocab) * b.k * es},
                 {b.xm, b.n * b.k * es}, {b.dz, b.n * (b.piece + kGap) * es}, {b.sums, b.dx.slices * a.rows * b.sums_ld * 4}}, b.bytes));
  }
  return true;
}

static bool gated(const fo_gated& a) {
  const int64_t es = (int64_t)elem_size(a.dtype);
  const GatedForward f = gated_forward(&a);
  CHECK(f.k >= a.cols && f.k * es % 128 == 0);
  CHECK(covers(f.c, a.features, a.rows, f.k * es / 128, true));
  CHECK(apart({{f.x, a.rows * f.k * es}, {f.gate, a.features * f.k * es}, {f.up, a.features * f.k * es}}, f.bytes));
  for (int need = 1; need < 4; ++need) {
    const bool dx = need & 1, dw = need & 2;
    const GatedBackward b = gated_backward(&a, dx, dw);
    CHECK(b.half % 64 == 0 && b.half >= a.features && 2 * b.half * es <= kMaxRowBytes);
    if (dx) CHECK(covers(b.dx, a.cols, a.rows, 2 * b.half * es / 128, false));
    if (dw) CHECK(covers(cut(a.dtype, a.cols, 2 * b.half, b.n * es / 128, false, true, false), a.cols, 2 * b.half, b.n * es / 128, false));
    CHECK(apart({{b.d, b.n * (2 * b.half + kGap) * es}, {b.x, a.rows * b.k * es}, {b.gate, a.features * b.k * es},
                 {b.up, a.features * b.k * es}, {b.sums, b.dx.slices * a.rows * b.sums_ld * 4}}, b.bytes));
  }
  return true;
}

int main() {
  std::mt19937_64 rng(7);
  auto size = [&](int bits) { return std::min<int64_t>(1 + (int64_t)(rng() >> (64 - 1 - rng() % bits)), (int64_t)1 << bits); };
  for (int trial = 0; trial < 20000; ++trial) {
    fo_loss a = {};
    do {
      a.rows = size(21); a.cols = size(20); a.vocab = size(24);
    } while (a.rows * a.cols > kMaxArea || a.rows * a.vocab > kMaxArea || a.cols * a.vocab > kMaxArea);
    a.dtype = rng() % 3;
    a.reduction = rng() % 3;
    a.smoothing = rng() % 2 ? 0.1 : 0.0;
    a.x = (const void*)(uintptr_t)(4096 + rng() % 2 * 4);
    a.weight = (const void*)(uintptr_t)(1 << 20);
    a.x_ld = a.cols + rng() % 3 * 4;
    a.weight_ld = a.cols + rng() % 2;
    if (!loss(a)) { printf("loss %ld %ld %ld type %d\n", (long)a.rows, (long)a.cols, (long)a.vocab, a.dtype); return 1; }
    fo_gated g = {};
    do {
      g.rows = size(21); g.cols = size(20); g.features = size(20);
    } while (g.rows * g.cols > kMaxArea || 2 * g.rows * g.features > kMaxArea || 2 * g.cols * g.features > kMaxArea);
    g.dtype = rng() % 3;
    g.x = g.gate = g.up = (const void*)(uintptr_t)4096;
    g.x_ld = g.cols;
    g.gate_ld = g.cols + rng() % 2;
    g.up_ld = g.cols;
    if (!gated(g)) { printf("gated %ld %ld %ld type %d\n", (long)g.rows, (long)g.cols, (long)g.features, g.dtype); return 1; }
  }
  // rows as they lie: whole steps, aligned, within the offsets
  if (!direct((void*)4096, 5, 64, 64, FO_BF16) || direct((void*)4098, 5, 64, 64, FO_BF16) || direct((void*)4096, 5, 63, 64, FO_BF16) ||
      direct((void*)4096, 5, 64, 65, FO_BF16) || !direct((void*)4096, 1, 64, 65, FO_BF16) || !direct((void*)4096, 5, 32, 32, FO_F32) ||
      direct((void*)4096, 5, 32, 32, FO_BF16) || direct((void*)4096, 2, 64, (int64_t)1 << 23, FO_BF16) || !direct((void*)4096, 9, 64, 0, FO_BF16)) {
    printf("direct\n");
    return 1;
  }
  printf("ok\n");
  return 0;
}
