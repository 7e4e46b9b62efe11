// fo_grads.hip -- the norm of many gradient tensors taken together, and clipping by
// it: kernels and C ABI (see include/foamd.h for the contract).
//
// Both are streams over a list of tensors: the norm reads every element once; clipping
// reads and writes them once more, and only where the norm passes the bound.  Nothing
// is done per tensor on the host but filling a table that goes to the kernels as an
// argument: no table is kept on the device, so calls may be captured and repeated.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "../../include/foamd.h"
#include "fo_error.hpp"
#include "fo_rows_args.hpp"
#include "fo_rows_device.hpp"

using namespace fo;
using rows::Bf16;
using rows::Fp16;
using rows::F32;
using rows::Chunk;

namespace {

#define FO_TRY(expr) do { const int rc_ = (expr); if (rc_) return rc_; } while (0)

// A tensor is cut into tiles of 16384 elements; tile boundaries depend on the list
// alone, and so do the sums' orders.
constexpr int kBlock = 512, kPer = 8, kTile = kBlock * kPer * 4;
// Workgroups of one call: 4 per compute unit, each of which takes consecutive tiles
// and writes one partial sum (a launch has one at least).
constexpr int64_t kGroups = 1024;
constexpr int kSums = 2048;                          // partial sums that a workspace holds
constexpr int64_t kWorkspace = kSums * (int64_t)sizeof(double);

// The tensors of one launch, as its argument (which may hold 4096 bytes).
// `first` is a tensor's first tile; `size` its elements, its types above bit 56.
template <int N, bool OUT>
struct Table {
  const void* grad[N];
  void* out[OUT ? N : 1];
  uint64_t size[N];
  uint32_t first[N];
  int count;
  uint32_t tiles;
};
constexpr int kInPlace = 196, kOutOfPlace = 140;
typedef Table<kInPlace, false> Plain;
typedef Table<kOutOfPlace, true> Paired;
static_assert(sizeof(Plain) <= 4000 && sizeof(Paired) <= 4000, "with a launch's other arguments: 4096 bytes");

constexpr uint64_t kSizeMask = (uint64_t(1) << 56) - 1;

template <typename T>
__device__ __forceinline__ void add_chunk(const Chunk<T>& c, int order, double& sum, uint32_t& top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = rows::elem<T>(c, i);
    if (order == FO_NORM_2) sum = __builtin_fma((double)f, (double)f, sum);
    else if (order == FO_NORM_1) sum += (double)fabsf(f);
    else top = max(top, __float_as_uint(f) & 0x7fffffffu);      // NaN patterns are above infinity's
  }
}

// A tile's loads are all on their way before the first is used.
template <typename T, int ORDER>
__device__ __forceinline__ void norm_tile(const void* grad, int64_t n, int64_t start, double& sum, uint32_t& top) {
  const typename T::raw* p = (const typename T::raw*)grad + start;
  const int64_t left = n - start;
  constexpr int PASSES = kTile / (kBlock * 8);
  Chunk<T> c[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t at = (int64_t)(i * kBlock + threadIdx.x) * 8;
    if (at < left) c[i] = rows::load_chunk<T>(p + at, (int)min(left - at, (int64_t)8));
    else
#pragma unroll
      for (int k = 0; k < rows::dwords<T>; ++k) c[i].w[k] = 0;
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) add_chunk<T>(c[i], ORDER, sum, top);
}

__device__ __forceinline__ double joined(double a, double b, int order) {
  if (order != FO_NORM_MAX) return a + b;
  const uint32_t x = __float_as_uint((float)a), y = __float_as_uint((float)b);       // both are floats >= 0 or NaN
  return (double)__uint_as_float(max(x & 0x7fffffffu, y & 0x7fffffffu));
}

// The sum over the workgroup, in lane 0 of wave 0 (every lane with `all`).
__device__ __forceinline__ double block_sum(double v, int order, double* lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = joined(v, __shfl_xor(v, d), order);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int i = 1; i < kBlock / 64; ++i) v = joined(v, lds[i], order);
  return v;
}

// The tensor of a tile: the last whose first tile is not past it.  Each lane compares
// a few entries (those past the last tensor are past every tile): one trip to memory
// instead of a binary search's eight.
template <int N, bool OUT>
__device__ __forceinline__ int tensor_of(const Table<N, OUT>& t, uint32_t tile) {
  int n = 0;
#pragma unroll
  for (int j = 0; j < (N + 63) / 64; ++j) {
    const int i = j * 64 + (int)(threadIdx.x & 63);
    n += __popcll(__ballot(i < N && t.first[min(i, N - 1)] <= tile));
  }
  return __builtin_amdgcn_readfirstlane(n - 1);
}

// One read of everything, squares summed in 64 bits (a product of two floats is exact
// there, and 2^40 terms lose nothing a float would show), in an order that the list alone
// decides.  Bound by memory: 1.745e9 floats 1.11 ms (6.3 TB/s, of the 7.1 that a bare
// read reaches), 124e6 bf16 38.7 us (6.4, partly from the memory-side cache), 25.6e6
// fp16 12 us.  Consecutive tiles per workgroup: with tiles dealt out in turn every tile
// needs its tensor looked up, 56 us instead of 40.  4096 workgroups gain nothing.
// Float32 by four elements per lane and access, as clipping reads it, took 1.89 ms.
template <int ORDER>
__global__ __launch_bounds__(kBlock) void k_grad_norm(Plain t, double* sums) {
  __shared__ double lds[kBlock / 64];
  const uint32_t begin = (uint32_t)((uint64_t)t.tiles * blockIdx.x / gridDim.x);
  const uint32_t end = (uint32_t)((uint64_t)t.tiles * (blockIdx.x + 1) / gridDim.x);
  double sum = 0.0;
  uint32_t top = 0;
  int i = tensor_of(t, begin);
  for (uint32_t tile = begin; tile < end; ++tile) {
    while (i + 1 < t.count && t.first[i + 1] <= tile) ++i;
    const int64_t n = (int64_t)(t.size[i] & kSizeMask), start = (int64_t)(tile - t.first[i]) * kTile;
    const int dtype = (int)(t.size[i] >> 56) & 3;
    if (dtype == FO_BF16) norm_tile<Bf16, ORDER>(t.grad[i], n, start, sum, top);
    else if (dtype == FO_FP16) norm_tile<Fp16, ORDER>(t.grad[i], n, start, sum, top);
    else norm_tile<F32, ORDER>(t.grad[i], n, start, sum, top);
  }
  if (ORDER == FO_NORM_MAX) sum = (double)__uint_as_float(top);
  sum = block_sum(sum, ORDER, lds);
  if (threadIdx.x == 0) ((FO_GLB double*)sums)[blockIdx.x] = sum;
}

// The norm from the partial sums, the same in every lane of every workgroup.
__device__ __forceinline__ double whole_norm(const double* sums, int count, int order, double* lds) {
  double v = 0.0;
  for (int i = threadIdx.x; i < count; i += kBlock) v = joined(v, ((const FO_GLB double*)sums)[i], order);
  v = block_sum(v, order, lds);
  return order == FO_NORM_2 ? sqrt(v) : v;
}

// min(1, max_norm / (norm + 1e-6)), as a float
__device__ __forceinline__ float clip_factor(double norm, double max_norm) {
  double q = max_norm / (norm + 1e-6);
  if (isinf(max_norm) || q > 1.0) q = 1.0;
  return (float)q;
}

// (`factor`: what clipping multiplies by, if not NULL)
__global__ __launch_bounds__(kBlock) void k_grad_norm_join(const double* sums, int count, int order, float* norm,
                                                           double max_norm, float* factor) {
  __shared__ double lds[kBlock / 64];
  const double v = whole_norm(sums, count, order, lds);
  if (threadIdx.x) return;
  *(FO_GLB float*)norm = (float)v;
  if (factor) *(FO_GLB float*)factor = clip_factor(v, max_norm);
}

// Float32 goes four elements per lane and access, so that a wave's access is one
// stretch of memory (a chunk of 8 would be two accesses 32 bytes apart).
template <typename O, int TILE>
__device__ __forceinline__ void clip_tile_f32(const void* grad, void* out, int64_t n, int64_t start, float c) {
  typedef uint32_t v2u __attribute__((ext_vector_type(2), aligned(2)));
  const float* p = (const float*)grad + start;
  typename O::raw* o = (typename O::raw*)out + start;
  const int64_t left = n - start;
  constexpr int PASSES = TILE / (kBlock * 4);
  rows::v4u in[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t at = (int64_t)(i * kBlock + threadIdx.x) * 4;
    if (at + 4 <= left) in[i] = *(const FO_GLB rows::v4u_a4*)(p + at);
    else
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at + k < left) in[i][k] = __float_as_uint(((const FO_GLB float*)p)[at + k]);
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t at = (int64_t)(i * kBlock + threadIdx.x) * 4;
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(in[i][k]) * c;
    if (at + 4 <= left) {
      if constexpr (rows::is_f32<O>) {
        const rows::v4u w = {__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
        *(FO_GLB rows::v4u_a4*)(o + at) = w;
      } else {
        const v2u w = {O::pack(f[0], f[1]), O::pack(f[2], f[3])};
        __builtin_nontemporal_store(w, (FO_GLB v2u*)(o + at));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at + k < left) {
          if constexpr (rows::is_f32<O>) ((FO_GLB float*)o)[at + k] = f[k];
          else ((FO_GLB uint16_t*)o)[at + k] = (uint16_t)O::pack(f[k], f[k]);
        }
    }
  }
}

template <typename T, typename O, int TILE>
__device__ __forceinline__ void clip_tile(const void* grad, void* out, int64_t n, int64_t start, float c) {
  if constexpr (rows::is_f32<T>) return clip_tile_f32<O, TILE>(grad, out, n, start, c);
  const typename T::raw* p = (const typename T::raw*)grad + start;
  typename O::raw* o = (typename O::raw*)out + start;
  const int64_t left = n - start;
  constexpr int PASSES = TILE / (kBlock * 8);
  Chunk<T> in[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t at = (int64_t)(i * kBlock + threadIdx.x) * 8;
    if (at < left) in[i] = rows::load_chunk<T>(p + at, (int)min(left - at, (int64_t)8));
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t at = (int64_t)(i * kBlock + threadIdx.x) * 8;
    if (at >= left) continue;
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = rows::elem<T>(in[i], k) * c;
    rows::store_chunk<O>(o + at, rows::to_chunk<O>(f), (int)min(left - at, (int64_t)8));
  }
}

template <typename T, int TILE>
__device__ __forceinline__ void clip_to(const void* grad, void* out, int out_dtype, int64_t n, int64_t start, float c) {
  if (out_dtype == FO_BF16) clip_tile<T, Bf16, TILE>(grad, out, n, start, c);
  else if (out_dtype == FO_FP16) clip_tile<T, Fp16, TILE>(grad, out, n, start, c);
  else clip_tile<T, F32, TILE>(grad, out, n, start, c);
}

// `TILE` elements from `start` on of the list's tensor i.
template <bool OUT, int TILE, typename Tab>
__device__ __forceinline__ void clip_part(const Tab& t, int i, int64_t start, float c) {
  const int64_t n = (int64_t)(t.size[i] & kSizeMask);
  const int dtype = (int)(t.size[i] >> 56) & 3;
  if constexpr (OUT) {
    const int od = (int)(t.size[i] >> 58) & 3;
    if (dtype == FO_BF16) clip_to<Bf16, TILE>(t.grad[i], t.out[i], od, n, start, c);
    else if (dtype == FO_FP16) clip_to<Fp16, TILE>(t.grad[i], t.out[i], od, n, start, c);
    else clip_to<F32, TILE>(t.grad[i], t.out[i], od, n, start, c);
  } else {
    void* g = const_cast<void*>(t.grad[i]);
    if (dtype == FO_BF16) clip_tile<Bf16, Bf16, TILE>(g, g, n, start, c);
    else if (dtype == FO_FP16) clip_tile<Fp16, Fp16, TILE>(g, g, n, start, c);
    else clip_tile<F32, F32, TILE>(g, g, n, start, c);
  }
}

struct ClipArgs { const double* sums; float* norm; double max_norm; int count, order, first; };

// Every workgroup joins the partial sums for itself (8 KB from L2: a launch less, and
// no workgroup waits for another).  Tiles go from the last to the first: what the norm
// read last is still in the memory-side cache.  Where the bound holds it ends here: 4.5
// us.  Scaling 2^30 bf16 elements in place takes 0.98 ms (4.4 TB/s).
template <typename Tab, bool OUT>
__global__ __launch_bounds__(kBlock) void k_grad_clip(Tab t, ClipArgs a) {
  __shared__ double lds[kBlock / 64];
  const double norm = whole_norm(a.sums, a.count, a.order, lds);
  if (a.first && blockIdx.x == 0 && threadIdx.x == 0) *(FO_GLB float*)a.norm = (float)norm;
  const float c = clip_factor(norm, a.max_norm);
  if (!OUT && c == 1.0f) return;
  const uint32_t begin = (uint32_t)((uint64_t)t.tiles * blockIdx.x / gridDim.x);
  const uint32_t end = (uint32_t)((uint64_t)t.tiles * (blockIdx.x + 1) / gridDim.x);
  if (begin == end) return;
  int i = tensor_of(t, end - 1);
  for (uint32_t tile = end; tile-- > begin;) {
    while (t.first[i] > tile) --i;
    clip_part<OUT, kTile>(t, i, (int64_t)(tile - t.first[i]) * kTile, c);
  }
}

// The same into other tensors, for lists past kPartsFrom tiles: half a tile per
// workgroup, the factor from k_grad_norm_join.  Workgroups that start and end as they
// come sweep through memory together, where 1024 ranges lie far apart: 1.745e9 elements
// float32 to bf16 take 1.76 ms (6.0 TB/s) against 2.05 (5.1); whole tiles 1.94, quarters
// 1.77.  One more launch, and grids that take time even to find nothing to do: 2^24
// elements gain nothing, and in place, where a norm within its bound is to cost no more
// than the norm, 2^30 bf16 elements took 0.21 ms less where they were scaled and
// 0.05 ms more where they were not, so that case keeps the kernel above.
constexpr int kParts = 2;
constexpr int64_t kPartsFrom = 4096;
constexpr uint32_t kPartsTo = uint32_t(1) << 21;     // of one launch, whose threads fit 32 bits
__global__ __launch_bounds__(kBlock) void k_grad_clip_parts(Paired t, const float* factor) {
  const float c = *(const FO_GLB float*)factor;
  const uint32_t part = gridDim.x - 1 - blockIdx.x, tile = part / kParts;
  const int i = tensor_of(t, tile);
  const int64_t start = (int64_t)(tile - t.first[i]) * kTile + part % kParts * (kTile / kParts);
  if (start < (int64_t)(t.size[i] & kSizeMask)) clip_part<true, kTile / kParts>(t, i, start, c);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
constexpr int32_t kMaxTensors = 1 << 17;
constexpr int64_t kMaxElems = int64_t(1) << 40;      // of one tensor

struct Span { uintptr_t lo, hi; bool out; };

int grad_checks(const fo_grad* list, int32_t count, int32_t order, const float* norm, const void* workspace, int64_t bytes,
                bool clip, int64_t* total) {
  if (count < 0 || count > kMaxTensors) return fail(FO_EINVAL, "count = %d is not in [0, 2^17]", (int)count);
  if (count && !list) return fail(FO_EINVAL, "list is NULL");
  if (order < FO_NORM_MAX || order > FO_NORM_2) return fail(FO_EINVAL, "bad norm order %d", (int)order);
  if (!norm || reinterpret_cast<uintptr_t>(norm) % 4) return fail(FO_EINVAL, "norm is NULL or not 4-byte aligned");
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || bytes < kWorkspace)
    return fail(FO_EINVAL, "the workspace must be 256-byte aligned and hold %lld bytes", (long long)kWorkspace);
  std::vector<Span> spans;
  if (clip) spans.reserve(2 * (size_t)count + 2);
  const uintptr_t norm_at = reinterpret_cast<uintptr_t>(norm), ws_at = reinterpret_cast<uintptr_t>(workspace);
  bool sorted = true, scratch = ws_at < norm_at + 4 && norm_at < ws_at + kWorkspace;
  auto add = [&](const void* p, int64_t n, bool out) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if ((uint64_t)n > UINTPTR_MAX - a) return false;
    const uintptr_t b = a + (uintptr_t)n;
    scratch |= (a < norm_at + 4 && norm_at < b) || (a < ws_at + kWorkspace && ws_at < b);
    if (clip) {                               // (what is only read may overlap)
      sorted &= spans.empty() || spans.back().lo <= a;
      spans.push_back({a, b, out});
    }
    return true;
  };
  *total = 0;
  for (int32_t i = 0; i < count; ++i) {
    const fo_grad& t = list[i];
    if (t.n < 0 || t.n > kMaxElems) return fail(FO_EINVAL, "tensor %d: n = %lld is not in [0, 2^40]", i, (long long)t.n);
    if (!rows::dtype_ok(t.dtype) || (clip && !rows::dtype_ok(t.out_dtype))) return fail(FO_EINVAL, "tensor %d: bad element type", i);
    if (t.n == 0) continue;
    const size_t es = rows::elem_size(t.dtype);
    if (!t.grad || reinterpret_cast<uintptr_t>(t.grad) % es) return fail(FO_EINVAL, "tensor %d: grad is NULL or misaligned", i);
    bool fits;
    if (clip) {
      const size_t os = rows::elem_size(t.out_dtype);
      if (!t.out || reinterpret_cast<uintptr_t>(t.out) % os) return fail(FO_EINVAL, "tensor %d: out is NULL or misaligned", i);
      if (t.out == t.grad) {
        if (t.dtype != t.out_dtype) return fail(FO_EINVAL, "tensor %d: clipped in place into another type", i);
        fits = add(t.grad, t.n * (int64_t)es, true);
      } else {
        fits = add(t.grad, t.n * (int64_t)es, false) && add(t.out, t.n * (int64_t)os, true);
      }
    } else {
      fits = add(t.grad, t.n * (int64_t)es, false);
    }
    if (!fits) return fail(FO_EINVAL, "tensor %d does not fit the address space", i);
    *total += (t.n + kTile - 1) / kTile;
  }
  if (scratch) return fail(FO_EALIAS, "the norm or the workspace overlaps a tensor of the list, or each other");
  if (!sorted) std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t hi_any = 0, hi_out = 0;
  for (const Span& s : spans) {
    if (s.lo < hi_out || (s.out && s.lo < hi_any)) return fail(FO_EALIAS, "arrays of the list overlap at %p", (void*)s.lo);
    hi_any = std::max(hi_any, s.hi);
    if (s.out) hi_out = std::max(hi_out, s.hi);
  }
  if (*total >> 31) return fail(FO_EINVAL, "the list holds more than 2^45 elements");
  return FO_OK;
}

int launch_check(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FO_OK : fail(FO_EHIP, "%s: %s", what, hipGetErrorString(e));
}

// Launches of at most N tensors each (those that `take` accepts), with their share of
// the workgroups.
template <int N, bool OUT, typename Take, typename Launch>
void each_table(const fo_grad* list, int32_t count, int64_t total, Take&& take, Launch&& launch) {
  Table<N, OUT> t;
  t.count = 0;
  t.tiles = 0;
  auto flush = [&] {
    if (!t.count) return;
    std::fill(t.first + t.count, t.first + N, UINT32_MAX);
    const int64_t share = (kGroups * t.tiles + total - 1) / total;
    launch(t, (unsigned)std::max<int64_t>(1, std::min<int64_t>(share, t.tiles)));
    t.count = 0;
    t.tiles = 0;
  };
  for (int32_t i = 0; i < count; ++i) {
    const fo_grad& g = list[i];
    if (g.n == 0 || !take(g)) continue;
    t.grad[t.count] = g.grad;
    if (OUT) t.out[t.count] = g.out;
    t.size[t.count] = (uint64_t)g.n | (uint64_t)g.dtype << 56 | (OUT ? (uint64_t)g.out_dtype << 58 : 0);
    t.first[t.count] = t.tiles;
    t.tiles += (uint32_t)((g.n + kTile - 1) / kTile);
    if (++t.count == N) flush();
  }
  flush();
}

// Partial sums of the list; their number.
int norm_launches(const fo_grad* list, int32_t count, int32_t order, int64_t total, double* sums, hipStream_t s) {
  int n = 0;
  each_table<kInPlace, false>(list, count, total, [](const fo_grad&) { return true; }, [&](const Plain& t, unsigned groups) {
    if (order == FO_NORM_2) hipLaunchKernelGGL(k_grad_norm<FO_NORM_2>, groups, kBlock, 0, s, t, sums + n);
    else if (order == FO_NORM_1) hipLaunchKernelGGL(k_grad_norm<FO_NORM_1>, groups, kBlock, 0, s, t, sums + n);
    else hipLaunchKernelGGL(k_grad_norm<FO_NORM_MAX>, groups, kBlock, 0, s, t, sums + n);
    n += (int)groups;
  });
  return n;
}
// a launch has at most its share, rounded up, so all have at most kGroups + one each
static_assert(kGroups + kMaxTensors / kInPlace + 1 < kSums, "the workspace holds every partial sum, and the factor");

}  // namespace

extern "C" {

int fo_grad_workspace(int64_t* bytes) {
  clear_error();
  if (!bytes) return fail(FO_EINVAL, "bytes is NULL");
  *bytes = kWorkspace;
  return FO_OK;
}

int fo_grad_norm(const fo_grad* list, int32_t count, int32_t order, float* norm, void* workspace, int64_t workspace_bytes,
                 void* stream) try {
  clear_error();
  int64_t total = 0;
  FO_TRY(grad_checks(list, count, order, norm, workspace, workspace_bytes, false, &total));
  hipStream_t s = static_cast<hipStream_t>(stream);
  double* sums = static_cast<double*>(workspace);
  const int n = norm_launches(list, count, order, total, sums, s);
  hipLaunchKernelGGL(k_grad_norm_join, 1, kBlock, 0, s, (const double*)sums, n, (int)order, norm, 0.0, (float*)nullptr);
  return launch_check("gradient norm launch");
} catch (const std::bad_alloc&) {
  return fail(FO_ENOMEM, "no host memory");
}

int fo_grad_clip(const fo_grad* list, int32_t count, int32_t order, double max_norm, float* norm, void* workspace,
                 int64_t workspace_bytes, void* stream) try {
  clear_error();
  if (!(max_norm >= 0.0)) return fail(FO_EINVAL, "max_norm must be >= 0");
  int64_t total = 0;
  FO_TRY(grad_checks(list, count, order, norm, workspace, workspace_bytes, true, &total));
  hipStream_t s = static_cast<hipStream_t>(stream);
  double* sums = static_cast<double*>(workspace);
  const int n = norm_launches(list, count, order, total, sums, s);
  ClipArgs a = {sums, norm, max_norm, n, (int)order, 1};
  float* factor = reinterpret_cast<float*>(sums + kSums - 1);
  auto join = [&](float* f) {
    hipLaunchKernelGGL(k_grad_norm_join, 1, kBlock, 0, s, (const double*)sums, n, (int)order, norm, max_norm, f);
    a.first = 0;
  };
  each_table<kInPlace, false>(list, count, total, [](const fo_grad& g) { return g.out == g.grad; },
                              [&](const Plain& t, unsigned groups) {
    hipLaunchKernelGGL((k_grad_clip<Plain, false>), groups, kBlock, 0, s, t, a);
    a.first = 0;
  });
  bool known = false;
  each_table<kOutOfPlace, true>(list, count, total, [](const fo_grad& g) { return g.out != g.grad; },
                                [&](const Paired& t, unsigned groups) {
    if (t.tiles >= kPartsFrom && t.tiles <= kPartsTo) {
      if (!known) join(factor);
      known = true;
      hipLaunchKernelGGL(k_grad_clip_parts, t.tiles * kParts, kBlock, 0, s, t, (const float*)factor);
    } else {
      hipLaunchKernelGGL((k_grad_clip<Paired, true>), groups, kBlock, 0, s, t, a);
    }
    a.first = 0;
  });
  if (a.first) join(nullptr);
  return launch_check("gradient clipping launch");
} catch (const std::bad_alloc&) {
  return fail(FO_ENOMEM, "no host memory");
}

}  // extern "C"
