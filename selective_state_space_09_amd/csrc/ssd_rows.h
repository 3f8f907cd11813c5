// Row access shared by the norm and step kernels: 8-element vectors of float32
// or bfloat16 rows with any alignment and any length, and the sum over the
// rows of a partial-sum table.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_device.h"

namespace ssd {

// 16 bytes at an address that is only element-aligned.  gfx950 takes
// unaligned global vector accesses, so a row of odd length needs no scalar
// path except for its last, partial vector.
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
struct Row8;

template <>
struct Row8<float> {
  u32x4_e4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const u32x4_e4*>(p);
    b = *reinterpret_cast<const u32x4_e4*>(p + 4);
  }
  // elements at and past n read as zero
  __device__ __forceinline__ void load_tail(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = i < n ? __float_as_uint(p[i]) : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = 4 + i < n ? __float_as_uint(p[4 + i]) : 0u;
  }
  __device__ __forceinline__ void zero() { a = 0u, b = 0u; }
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(i < 4 ? a[i] : b[i - 4]);
  }
  __device__ __forceinline__ static void store(float* p, const float* f) {
    u32x4_e4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(f[i]), b[i] = __float_as_uint(f[4 + i]);
    *reinterpret_cast<u32x4_e4*>(p) = a;
    *reinterpret_cast<u32x4_e4*>(p + 4) = b;
  }
  __device__ __forceinline__ static void store1(float* p, float f) { *p = f; }
};

template <>
struct Row8<uint16_t> {
  u32x4_e2 a;
  __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const u32x4_e2*>(p); }
  __device__ __forceinline__ void load_tail(const uint16_t* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < n ? p[2 * i] : 0u, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0u;
      a[i] = lo | hi << 16;
    }
  }
  __device__ __forceinline__ void zero() { a = 0u; }
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(i & 1 ? a[i >> 1] & 0xFFFF0000u : a[i >> 1] << 16);
  }
  __device__ __forceinline__ static void store(uint16_t* p, const float* f) {
    u32x4_e2 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<u32x4_e2*>(p) = a;
  }
  __device__ __forceinline__ static void store1(uint16_t* p, float f) {
    *p = static_cast<uint16_t>(pack_bf16x2(f, 0.0f) & 0xFFFFu);
  }
};

// vector v (elements 8v .. 8v+7) of a row of L elements
template <typename T>
__device__ __forceinline__ Row8<T> row_load(const T* row, int v, int L) {
  Row8<T> r;
  const int n = L - 8 * v;
  if (n >= 8)
    r.load(row + 8 * v);
  else if (n > 0)
    r.load_tail(row + 8 * v, n);
  else
    r.zero();
  return r;
}
template <typename T>
__device__ __forceinline__ void row_store(T* row, int v, int L, const float* f) {
  const int n = L - 8 * v;
  if (n >= 8) {
    Row8<T>::store(row + 8 * v, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) Row8<T>::store1(row + 8 * v + i, f[i]);
  }
}

// out[j] = sum over the nparts rows of part (nparts, n), j < n; columns
// [0, na) go to a, the rest to b.  Fixed order: no atomics, so the same inputs
// give the same bits.
hipError_t sum_parts(const float* part, int nparts, int n, float* a, int na, float* b,
                     hipStream_t st);

}  // namespace ssd
