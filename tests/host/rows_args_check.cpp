// The host half of the row operators' launcher (csrc/fo_rows_args.hpp) against
// brute force: extents and overlap of strided arrays, 64-bit limits, and that
// every spread covers its row and every workspace its partial sums.
#include <cstdarg>
#include <cstdio>
#include <random>
#include <set>

#include "../../precision_optimizer_state_amd/csrc/fo_rows_args.hpp"

int fo::fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return code;
}
void fo::clear_error() {}

using namespace fo::rows;

#define CHECK(c)                                                     \
  do {                                                               \
    if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return 1; }   \
  } while (0)

static const void* at(uint64_t a) { return reinterpret_cast<const void*>(a); }

int main() {
  std::mt19937_64 rng(5);
  auto pick = [&](int n) { return (int64_t)(rng() % n); };

  // overlap: spans [first, last] byte touched, by enumeration of the end rows
  for (int trial = 0; trial < 200000; ++trial) {
    Arrays a;
    struct Want { uint64_t lo, hi; bool out; } want[4];
    bool overlap = false;
    for (int i = 0; i < 4; ++i) {
      const size_t size = pick(2) ? 2 : 4;
      const int64_t rows = 1 + pick(4), cols = 1 + pick(9), ld = pick(3) ? cols + pick(5) : pick(3);
      const uint64_t base = 4096 + (uint64_t)pick(200) * size;
      const bool out = pick(2);
      CHECK(a.add(at(base), "a", out, true, rows, cols, ld, size) == FO_OK);
      uint64_t hi = 0;
      for (int64_t r = 0; r < rows; ++r) hi = std::max<uint64_t>(hi, base + (uint64_t)(r * ld + cols) * size);
      want[i] = {base, hi, out};
      for (int j = 0; j < i; ++j)
        overlap |= (want[j].out || out) && want[j].lo < hi && base < want[j].hi;
    }
    CHECK((a.disjoint() == FO_EALIAS) == overlap);
  }

  // refusals and the ends of the 64-bit range
  Arrays a;
  CHECK(a.add(nullptr, "a", false, true, 1, 1, 1, 2) == FO_EINVAL && a.add(nullptr, "a", false, false, 1, 1, 1, 2) == FO_OK);
  CHECK(a.add(at(4097), "a", false, true, 1, 1, 1, 2) == FO_EINVAL && a.add(at(4098), "a", false, true, 1, 1, 1, 4) == FO_EINVAL);
  CHECK(a.add(at(4096), "a", false, true, 2, 1, -1, 2) == FO_EINVAL);
  CHECK(a.add(at(4096), "a", false, true, kMaxRows, kMaxCols, INT64_MAX, 4) == FO_EINVAL);
  CHECK(a.add(at(4096), "a", false, true, kMaxRows, kMaxCols, 0, 4) == FO_OK);
  CHECK(a.add(at(UINT64_MAX - 63), "a", false, true, 1, 64, 64, 2) == FO_EINVAL);
  CHECK(a.n == 1);
  CHECK(a.add(at(4096), "a", true, true, 0, 64, 64, 2) == FO_OK && a.n == 1);      // no rows: nothing is touched

  // spreads: every chunk of the row has a lane, thread counts are whole teams
  std::set<int64_t> sizes = {kMaxCols, kMaxCols - 1};
  for (int64_t c = 1; c < 20000; ++c) sizes.insert(c);
  for (int64_t cols : sizes) {
    const int64_t n = (cols + 7) / 8;
    const Spread f = fwd_spread(cols);
    CHECK(f.lanes == 0 ? n > 2048 : (int64_t)f.lanes * f.chunks >= n && fwd_threads(f.lanes) % f.lanes == 0);
    for (int call = 0; call < 6; ++call) {
      const int dt = call % 3;
      const bool dropping = call >= 3;
      const Spread b = bwd_spread(cols, dt, dropping);
      CHECK(b.lanes == 0 ? n > (dt == FO_F32 || dropping ? 1024 : 2048) : (int64_t)b.lanes * b.chunks >= n && kBwdThreads % b.lanes == 0);
      for (int64_t rows : {int64_t(0), int64_t(1), int64_t(7), int64_t(1000), int64_t(1) << 24, kMaxRows}) {
        const int64_t s = bwd_splits(rows, cols, dt, dropping);
        CHECK(rows == 0 ? s == 0 : s >= 1 && s <= kColGroups);
        CHECK(2 * s * cols * 4 <= bwd_workspace(rows, cols));
        if (b.lanes) CHECK(s <= kBwdGroups && (s == kBwdGroups || s * (kBwdThreads / b.lanes) >= rows));
      }
    }
  }
  CHECK(shape_ok(0, 1) == FO_OK && shape_ok(kMaxRows, kMaxCols) == FO_OK);
  CHECK(shape_ok(-1, 1) && shape_ok(kMaxRows + 1, 1) && shape_ok(1, 0) && shape_ok(1, kMaxCols + 1));
  printf("ok\n");
  return 0;
}
