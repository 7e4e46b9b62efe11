// fo_rows_args.hpp -- host-only half of the row operators' launcher: limits,
// argument extents and overlap, and how rows are spread over a launch.  No HIP:
// tests/host/rows_args_check.cpp compiles it alone.
#pragma once

#include <stdint.h>
#include <stddef.h>

#include <algorithm>

#include "../../include/foamd.h"
#include "fo_error.hpp"

namespace fo {
namespace rows {

constexpr int64_t kMaxCols = int64_t(1) << 26;     // of norms: k_norm_bwd_reduce takes 32 threads per column
constexpr int64_t kMaxDropCols = int64_t(1) << 40;
constexpr int64_t kMaxRows = int64_t(1) << 40;

inline size_t elem_size(int dtype) { return dtype == FO_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == FO_BF16 || dtype == FO_FP16 || dtype == FO_F32; }

inline int rows_ok(int64_t rows) {
  return rows < 0 || rows > kMaxRows ? fail(FO_EINVAL, "rows = %lld is not in [0, 2^40]", (long long)rows) : FO_OK;
}
inline int shape_ok(int64_t rows, int64_t cols) {
  if (const int rc = rows_ok(rows)) return rc;
  if (cols < 1 || cols > kMaxCols) return fail(FO_EINVAL, "cols = %lld is not in [1, 2^26]", (long long)cols);
  return FO_OK;
}
inline int drop_shape_ok(int64_t rows, int64_t cols) {
  if (const int rc = rows_ok(rows)) return rc;
  if (cols < 1 || cols > kMaxDropCols) return fail(FO_EINVAL, "cols = %lld is not in [1, 2^40]", (long long)cols);
  return FO_OK;
}

// The smallest k with 4^k >= cols (see FwdArgs)
inline int quarter_log(int64_t cols) {
  int k = 0;
  while ((int64_t(1) << 2 * k) < cols) ++k;
  return k;
}

// The arrays of one call: checked one by one, then the outputs against all.
struct Arrays {
  struct Span { uintptr_t lo, hi; bool out; const char* name; };
  Span s[16];
  int n = 0;

  // `rows` rows of `cols` elements of `size` bytes, `ld` elements apart
  int add(const void* p, const char* name, bool out, bool required, int64_t rows, int64_t cols, int64_t ld, size_t size,
          size_t align = 0) {
    if (!p) return required ? fail(FO_EINVAL, "%s is NULL", name) : FO_OK;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a % (align ? align : size)) return fail(FO_EINVAL, "%s is not %zu-byte aligned", name, align ? align : size);
    if (ld < 0) return fail(FO_EINVAL, "the row stride of %s is negative", name);
    const unsigned __int128 bytes = ((unsigned __int128)(rows > 0 ? rows - 1 : 0) * (uint64_t)ld + (uint64_t)cols) * size;
    if (bytes > (unsigned __int128)(UINTPTR_MAX - a) || bytes >> 62)
      return fail(FO_EINVAL, "%s does not fit the address space", name);
    if (rows > 0) s[n++] = {a, a + (uintptr_t)bytes, out, name};
    return FO_OK;
  }

  int disjoint() const {
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j)
        if ((s[i].out || s[j].out) && s[i].lo < s[j].hi && s[j].lo < s[i].hi)
          return fail(FO_EALIAS, "%s and %s overlap", s[i].name, s[j].name);
    return FO_OK;
  }
};

// How a row is spread over lanes: `lanes` of them with `chunks` 8-element chunks
// each, or lanes = 0 for rows that do not fit registers (k_norm_*_long).
struct Spread { int lanes, chunks; };

// Forward: the fewest lanes that cover the row with up to two chunks each, and
// three between 512 and 768 columns, where 64 lanes of two leave up to half of
// them idle (131072 rows of 520 columns bf16, layer norm 54.1 us against 61.5, with
// dropout and residual 111 against 119; of 640 columns 56.5 against 64.6 and 114
// against 125; of 768, where it is a quarter, 68.9 against 69.5 and 139 against 135,
// and at 8192 rows 6.2 against 6.4 and 10.8 against 11.1).  Float32 rows lose 5% by
// it (RMS norm of 32768 x 640, 40.3 us against 38.1).
inline Spread fwd_spread(int64_t cols) {
  const int64_t n = (cols + 7) / 8;
  if (n <= 8) return {8, 1};
  if (n > 64 && n <= 96) return {32, 3};
  for (int lanes = 8; lanes <= 1024; lanes *= 2)
    if (n <= 2 * lanes) return {lanes, 2};
  return {0, 0};
}

// Backward: one chunk per lane (see k_norm_bwd), two where 1024 lanes of one do
// not reach, against the kernels of long rows, last sums included: 1024 x 16384 bf16
// layer norm 36.4 us against 45.6, with residual (which spills 5 registers) 44.6
// against 52.0; 1024 x 8200, 24.0 against 27.9 and 29.5 against 33.3.  Two of float32,
// or two with dropout, do not fit the registers of 1024 threads: 1024 x 16384 bf16
// with residual and dropout takes 67.3 us so, 58.1 with the kernels of long rows.
inline Spread bwd_spread(int64_t cols, int dtype, bool dropping) {
  const int64_t n = (cols + 7) / 8;
  for (int lanes = 8; lanes <= 1024; lanes *= 2)
    if (n <= lanes) return {lanes, 1};
  if (n <= 2048 && dtype != FO_F32 && !dropping) return {1024, 2};
  return {0, 0};
}

constexpr int fwd_threads(int lanes) { return std::max(lanes, 256); }
constexpr int kBwdThreads = 1024;

// Workgroups of the backward kernels: one per compute unit, each of which writes
// one partial sum per weight gradient.  A constant, so that the order of those
// sums is the same on every device.
constexpr int64_t kBwdGroups = 256;
constexpr int64_t kColGroups = 2048;        // of k_norm_bwd_cols_long, over columns and ranges of rows

inline int64_t bwd_splits(int64_t rows, int64_t cols, int dtype, bool dropping) {
  const Spread s = bwd_spread(cols, dtype, dropping);
  if (s.lanes) return std::min<int64_t>((rows * s.lanes + kBwdThreads - 1) / kBwdThreads, kBwdGroups);
  return std::min<int64_t>((rows + 7) / 8, std::max<int64_t>(kColGroups / ((cols + 255) / 256), 1));
}

// Bytes of workspace: two partial sums per column, of the call that needs the
// most ranges of rows.
inline int64_t bwd_workspace(int64_t rows, int64_t cols) {
  int64_t splits = 0;
  for (int dtype : {(int)FO_BF16, (int)FO_FP16, (int)FO_F32})
    for (bool dropping : {false, true}) splits = std::max(splits, bwd_splits(rows, cols, dtype, dropping));
  return 2 * splits * cols * (int64_t)sizeof(float);
}

}  // namespace rows
}  // namespace fo
