// fo_rows_device.hpp -- device helpers of the row operators (dropout, layer
// norm, RMS norm and their fused form): 8-element chunks of rows in any of the
// three element types, and the counter-based keep decisions of dropout.
//
// A row of C elements is cut into ceil(C / 8) chunks.  A chunk is what one lane
// holds (16 bytes of a 16-bit type) and what one generator call decides, so a
// lane never needs its neighbour's words and any kernel that holds chunks finds
// the same mask, whatever its launch shape.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fo {
namespace rows {

#define FO_GLB __attribute__((address_space(1)))
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
// Rows of an odd length begin at any element, so vector accesses only claim
// the element's alignment; gfx950 serves unaligned 16-byte global accesses
// itself (one instruction either way), aligned ones at no extra cost.
typedef v4u v4u_a2 __attribute__((aligned(2)));
typedef v4u v4u_a4 __attribute__((aligned(4)));

struct Bf16 {
  typedef uint16_t raw;
  typedef v4u_a2 vec;
  static __device__ __forceinline__ float widen(uint32_t h) { return __uint_as_float(h << 16); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {    // one RNE conversion each
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
  }
};
struct Fp16 {
  typedef uint16_t raw;
  typedef v4u_a2 vec;
  static __device__ __forceinline__ float widen(uint32_t h) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
           (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
  }
};
struct F32 {
  typedef float raw;
  typedef v4u_a4 vec;
};
template <typename T> constexpr bool is_f32 = false;
template <> inline constexpr bool is_f32<F32> = true;
template <typename T> constexpr int dwords = is_f32<T> ? 8 : 4;     // of one chunk

// One chunk as loaded (still in its type).
template <typename T> struct Chunk { uint32_t w[dwords<T>]; };

template <typename T>
__device__ __forceinline__ float elem(const Chunk<T>& c, int i) {
  if constexpr (is_f32<T>) return __uint_as_float(c.w[i]);
  else return T::widen(i & 1 ? c.w[i >> 1] >> 16 : c.w[i >> 1] & 0xffffu);
}

template <typename T>
__device__ __forceinline__ Chunk<T> to_chunk(const float* f) {
  Chunk<T> c;
#pragma unroll
  for (int i = 0; i < dwords<T>; ++i) {
    if constexpr (is_f32<T>) c.w[i] = __float_as_uint(f[i]);
    else c.w[i] = T::pack(f[2 * i], f[2 * i + 1]);
  }
  return c;
}

// cnt (>= 1) valid elements at p; the rest of the chunk reads as 0 and nothing
// past the valid ones is touched.
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const typename T::raw* ptr, int cnt) {
  const FO_GLB typename T::raw* p = (const FO_GLB typename T::raw*)ptr;
  Chunk<T> c;
  if (cnt >= 8) {
#pragma unroll
    for (int q = 0; q < dwords<T> / 4; ++q) {
      const v4u v = ((const FO_GLB typename T::vec*)p)[q];
#pragma unroll
      for (int i = 0; i < 4; ++i) c.w[4 * q + i] = v[i];
    }
    return c;
  }
#pragma unroll
  for (int i = 0; i < dwords<T>; ++i) c.w[i] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < cnt) {
      if constexpr (is_f32<T>) c.w[i] = __float_as_uint(p[i]);
      else c.w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  return c;
}

// Stores of 16-bit chunks carry the nontemporal hint unless the kernel that writes
// them reads them back (REREAD: h in k_norm_fwd_long).  Measured on an RMS norm of
// 8192 x 4096 bf16: 24.9 -> 20.0 us (the time of a plain copy); the hint on the
// loads as well took it to 24.4.  What is read back loses by it: residual + layer
// norm of 838 x 20000 bf16, 46.6 us against 41.8.  A float32 chunk is two stores 32
// bytes apart from the next lane's, which a plain store joins in cache: layer norm
// backward 32768 x 2048, 150 us against 160 with the hint.
template <typename T, bool REREAD = false>
__device__ __forceinline__ void store_chunk(typename T::raw* ptr, const Chunk<T>& c, int cnt) {
  FO_GLB typename T::raw* p = (FO_GLB typename T::raw*)ptr;
  if (cnt >= 8) {
#pragma unroll
    for (int q = 0; q < dwords<T> / 4; ++q) {
      const v4u v = {c.w[4 * q], c.w[4 * q + 1], c.w[4 * q + 2], c.w[4 * q + 3]};
      if constexpr (is_f32<T> || REREAD) ((FO_GLB typename T::vec*)p)[q] = v;
      else __builtin_nontemporal_store(v, (FO_GLB typename T::vec*)p + q);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < cnt) {
      if constexpr (is_f32<T>) p[i] = __uint_as_float(c.w[i]);
      else p[i] = (uint16_t)(c.w[i >> 1] >> (16 * (i & 1)));
    }
}

// A chunk of a row that begins at column `col`, in two steps, so that the loads
// of several arrays are all on their way before any result is touched (a lane
// that gathers a short last chunk element by element waits for each array in
// turn: 4096 x 4095 bf16 layer norm, 17.4 and 31.6 us forward and backward so,
// against 12.6 and 19.6 at 4096 columns).  load_part reads the last chunk of a
// row that is no multiple of 8 long as the row's last 8 elements; settle_part
// moves its own elements down and clears the rest.  Rows of fewer than 8
// elements are gathered.  Nothing outside the row is read; a chunk past its end
// is 0.
template <typename T>
__device__ __forceinline__ Chunk<T> load_part(const typename T::raw* row, int col, int cols) {
  Chunk<T> c;
  if (cols < 8 && col < cols) return load_chunk<T>(row + col, cols - col);
  if (col < cols) return load_chunk<T>(row + min(col, cols - 8), 8);
#pragma unroll
  for (int i = 0; i < dwords<T>; ++i) c.w[i] = 0;
  return c;
}

template <typename T>
__device__ __forceinline__ void settle_part(Chunk<T>& c, int col, int cols) {
  const int k = col + 8 - cols;                    // elements of the chunk before
  if (cols < 8 || k <= 0 || k >= 8) return;
  constexpr int N = dwords<T>;
#pragma unroll
  for (int step = N / 2; step; step >>= 1)         // whole dwords
    if (k & (is_f32<T> ? step : 2 * step)) {
#pragma unroll
      for (int i = 0; i < N; ++i) c.w[i] = i + step < N ? c.w[i + step] : 0;
    }
  if constexpr (!is_f32<T>)
    if (k & 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) c.w[i] = c.w[i] >> 16 | (i + 1 < N ? c.w[i + 1] << 16 : 0);
    }
}

// Norm weights and biases come in any of the three types, whatever the rows
// hold; a branch on a kernel argument picks the load.  NULL reads as `fill`.
enum { DT_BF16 = 0, DT_FP16 = 1, DT_F32 = 2 };

__device__ __forceinline__ void load_param(const void* base, int dt, int64_t col, int cnt, float fill, float* f) {
  if (!base) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fill;
  } else if (dt == DT_F32) {
    const Chunk<F32> c = load_chunk<F32>((const float*)base + col, cnt);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = elem<F32>(c, i);
  } else if (dt == DT_BF16) {
    const Chunk<Bf16> c = load_chunk<Bf16>((const uint16_t*)base + col, cnt);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = elem<Bf16>(c, i);
  } else {
    const Chunk<Fp16> c = load_chunk<Fp16>((const uint16_t*)base + col, cnt);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = elem<Fp16>(c, i);
  }
}

__device__ __forceinline__ void store_param(void* base, int dt, int64_t col, float f) {
  if (dt == DT_F32) ((FO_GLB float*)base)[col] = f;
  else if (dt == DT_BF16) ((FO_GLB uint16_t*)base)[col] = (uint16_t)Bf16::pack(f, f);
  else ((FO_GLB uint16_t*)base)[col] = (uint16_t)Fp16::pack(f, f);
}

// ---------------------------------------------------------------------------
// dropout's keep decisions
// ---------------------------------------------------------------------------
// Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64-bit
// products over a 128-bit counter under a 64-bit key.  The counter is (chunk
// index, offset), the key the seed.
//
// Element j of a chunk owns half-word j of the chunk's first four words as the
// high 16 bits of a 32-bit uniform u, and half-word j of a second call (bit 63
// of the chunk index set) as the low 16 bits; it is kept where u >= thr.  The
// high half decides unless it equals thr's (once in 2^16 elements), so the
// second call runs only in chunks where some lane needs it: one generator call
// per 8 elements instead of two, with the drop rate held to 2^-32.  Measured on
// 2^25 bf16 elements: 20.3-22.4 us (5.9-6.6 TB/s, the time of the copy without
// a mask) against 26.2 us for two calls per chunk.
struct DropArgs {
  uint32_t thr;          // round(2^32 p)
  float scale;           // 1 / (1 - thr / 2^32)
  int all;               // p rounds to 1: everything is dropped
  uint64_t seed, offset;
  const uint64_t* state; // NULL, or {seed, offset} to add (read on the device)
};

struct DropKey { uint32_t k0, k1, o0, o1; };

__device__ __forceinline__ DropKey drop_key(const DropArgs& d) {
  uint64_t s = d.seed, o = d.offset;
  if (d.state) { s += ((const FO_GLB uint64_t*)d.state)[0]; o += ((const FO_GLB uint64_t*)d.state)[1]; }
  return {(uint32_t)s, (uint32_t)(s >> 32), (uint32_t)o, (uint32_t)(o >> 32)};
}

__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, const DropKey& k, uint32_t* w) {
  uint32_t c2 = k.o0, c3 = k.o1, k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0; w[1] = c1; w[2] = c2; w[3] = c3;
}

__device__ __forceinline__ uint32_t half_of(const uint32_t* w, int j) {
  return j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
}

// f[j] = kept ? f[j] / (1 - p) : 0 for the 8 elements of chunk `index`
__device__ __forceinline__ void drop_chunk(const DropArgs& d, const DropKey& k, uint64_t index, float* f) {
  if (d.all) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] *= d.scale;
  uint32_t w[4];
  philox((uint32_t)index, (uint32_t)(index >> 32), k, w);
  const uint32_t hi = d.thr >> 16, lo = d.thr & 0xffffu;
  bool open = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) open |= half_of(w, j) == hi;
  if (open && lo != 0) {
    uint32_t v[4];
    philox((uint32_t)index, (uint32_t)(index >> 32) | 0x80000000u, k, v);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (((half_of(w, j) << 16) | half_of(v, j)) < d.thr) f[j] = 0.0f;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (half_of(w, j) < hi) f[j] = 0.0f;
}

}  // namespace rows
}  // namespace fo
