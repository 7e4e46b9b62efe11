// More of the products' host half (csrc/fo_products_args.hpp) against brute force: where
// the backward pass of the loss keeps the statistics that it makes again, float32 sums of
// long k, and the threads of a launch.
#include <cstdarg>
#include <cstdio>
#include <random>

#include "../../precision_optimizer_state_amd/csrc/fo_products_args.hpp"

int fo::fail(int code, const char*, ...) { return code; }
void fo::clear_error() {}

using namespace fo::prod;

#define CHECK(c)                                                     \
  do {                                                               \
    if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return false; } \
  } while (0)

static bool loss(const fo_loss& a) {
  const int64_t es = (int64_t)elem_size(a.dtype);
  const LossForward f = loss_forward(&a);
  for (int need = 1; need < 4; ++need) {
    const LossBackward b = loss_backward(&a, need & 1, need & 2);
    // the same tiles as the forward pass's, and pieces that end where tiles do
    CHECK(b.k == f.k && b.statistics.kind == f.c.kind && b.statistics.tiles_r == f.c.tiles_r && b.statistics.tiles_c == f.c.tiles_c);
    CHECK(b.piece >= a.vocab || b.piece % 256 == 0);
    int64_t tiles = 0;
    for (int64_t first = 0; first < a.vocab; first += b.piece) {
      const int64_t nv = std::min(b.piece, a.vocab - first), tile = tile_r(b.statistics.kind);
      CHECK(first / tile == tiles);
      tiles += (nv + tile - 1) / tile;
      // the logits again: the same kind of tile, each of which begins at a token that is there, and
      // which reach all tokens' whole steps (a narrow one writes its step's other half itself)
      const Cut c = b.logits(nv, a.rows);
      CHECK(c.kind == f.c.kind && c.slices == 1 && c.tiles_r == (nv + tile - 1) / tile);
      CHECK((int64_t)(c.tiles_c - 1) * tile_c(c.kind) < a.rows);
      CHECK(c.kind == NARROW ? a.rows <= 32 && b.n == 64 && c.tiles_c == 1 : (int64_t)c.tiles_c * tile_c(c.kind) >= b.n);
      CHECK((__int128)c.tiles_r * c.tiles_c * threads(c.kind) < ((__int128)1 << 32));
    }
    CHECK(tiles == f.c.tiles_r && b.parts == tiles * waves_r(f.c.kind));
    // (gradients of logits take that place afterwards)
    const int64_t dz_end = b.sums >= 0 ? b.sums : b.bytes;
    CHECK(b.part == b.dz && b.part + b.parts * a.rows * 8 <= dz_end && b.dz + b.n * (b.piece + kGap) * es <= dz_end);
    // the rest, and what lies before and behind it
    CHECK(b.rest >= 0 && b.rest % 256 == 0 && b.rest + a.rows * 4 <= b.dz);
    CHECK(b.factor < 0 || (b.unit + a.rows * 4 <= b.factor && b.factor + 4 <= b.rest));
    CHECK(b.x < 0 || b.x + a.rows * b.k * es <= b.rest);
    CHECK(b.w < 0 || b.w + std::min(b.piece, a.vocab) * b.k * es <= b.rest);
    CHECK(b.xm < 0 || b.xm + b.n * b.k * es <= b.rest);
  }
  return true;
}

// Wide tiles' float32 sums are one chain each: of at most 64 steps, 2048 terms.
static bool chains(int64_t nr, int64_t nc, int64_t steps) {
  for (int form = 0; form < 8; ++form) {
    const Cut c = cut(FO_F32, nr, nc, steps, form & 1, form & 2, form & 4);
    CHECK(c.slices >= 1 && (c.kind != WIDE || (steps + c.slices - 1) / c.slices <= 64));
  }
  return true;
}

// A launch's threads and workgroups are 32-bit numbers.
static bool fits(int dtype, int64_t nr, int64_t nc, int64_t steps) {
  for (int form = 0; form < 8; ++form) {
    const Cut c = cut(dtype, nr, nc, steps, form & 1, form & 2, form & 4);
    const __int128 groups = (__int128)c.tiles_r * c.tiles_c * c.slices;
    CHECK(groups >= 1 && groups < ((__int128)1 << 31) && groups * threads(c.kind) < ((__int128)1 << 32));
  }
  return true;
}

int main() {
  std::mt19937_64 rng(11);
  auto size = [&](int bits) { return std::min<int64_t>(1 + (int64_t)(rng() >> (64 - 1 - rng() % bits)), (int64_t)1 << bits); };
  for (int trial = 0; trial < 10000; ++trial) {
    fo_loss a = {};
    do {
      a.rows = size(21); a.cols = size(20); a.vocab = size(24);
    } while (a.rows * a.cols > kMaxArea || a.rows * a.vocab > kMaxArea || a.cols * a.vocab > kMaxArea);
    a.dtype = rng() % 3;
    a.reduction = rng() % 3;
    a.x = a.weight = (const void*)(uintptr_t)(4096 + rng() % 2 * 4);
    a.x_ld = a.cols + rng() % 3 * 4;
    a.weight_ld = a.cols + rng() % 2;
    const int64_t steps = size(16);
    if (!chains(a.vocab, a.rows, steps)) { printf("%ld x %ld, %ld steps\n", (long)a.vocab, (long)a.rows, (long)steps); return 1; }
    if (!loss(a)) { printf("loss %ld %ld %ld type %d\n", (long)a.rows, (long)a.cols, (long)a.vocab, a.dtype); return 1; }
  }
  // any two sizes that the limits allow, at and around powers of two
  for (int dtype = 0; dtype < 3; ++dtype)
    for (int r = 0; r <= 24; ++r)
      for (int c = 0; c <= 24 && r + c <= 36; ++c)
        for (int64_t odd : {-1, 0, 1})
          for (int64_t steps : {1, 2, 11, 12, 64, 65, 1000, 1 << 15, 1 << 16}) {
            const int64_t nr = std::max<int64_t>(1, ((int64_t)1 << r) + odd), nc = (int64_t)1 << c;
            if (nr * nc > kMaxArea) continue;
            if (!fits(dtype, nr, nc, steps) || !fits(dtype, nc, nr, steps)) {
              printf("%ld x %ld, %ld steps, type %d\n", (long)nr, (long)nc, (long)steps, dtype);
              return 1;
            }
          }
  printf("ok\n");
  return 0;
}
