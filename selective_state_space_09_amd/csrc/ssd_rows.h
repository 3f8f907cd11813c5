// Row access shared by the norm and step kernels: 8-element vectors of float32
// or bfloat16 rows with any alignment and any length, and the sum over the
// rows of a partial-sum table.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_device.h"

namespace ssd {

// 16 bytes at an address that is only element-aligned.  gfx950 takes
// unaligned global vector accesses, so rows of odd length or stride need no
// scalar path.
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));

// eight consecutive elements of a row
template <typename T>
struct Row8;

template <>
struct Row8<float> {
  u32x4_e4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const u32x4_e4*>(p);
    b = *reinterpret_cast<const u32x4_e4*>(p + 4);
  }
  // the n < 8 elements of a row shorter than a vector; zeros behind them
  __device__ __forceinline__ void load_short(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = i < n ? __float_as_uint(p[i]) : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = 4 + i < n ? __float_as_uint(p[4 + i]) : 0u;
  }
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
  __device__ __forceinline__ void load_short(const uint16_t* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < n ? p[2 * i] : 0u, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0u;
      a[i] = lo | hi << 16;
    }
  }
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

// Where HIDE, hides where a value comes from: the compiler neither keeps what it
// loaded through p (a weight row, the same for every row of a loop) nor what it
// made of r in registers from one use to the next, which with several vectors a
// lane costs the waves that hide the latency of the rows.  With one vector the
// registers are there and the work is saved (gated norm backward, 4096 x 4096 in
// 8 groups: 34.3 us, made and loaded again 38.8).
template <bool HIDE, typename T>
__device__ __forceinline__ const T* reload(const T* p) {
  if constexpr (HIDE) asm volatile("" : "+s"(p));
  return p;
}
template <bool HIDE>
__device__ __forceinline__ void remake(Row8<float>& r) {
  if constexpr (HIDE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a = r.a[i], b = r.b[i];
      asm volatile("" : "+v"(a), "+v"(b));
      r.a[i] = a, r.b[i] = b;
    }
  }
}
template <bool HIDE>
__device__ __forceinline__ void remake(Row8<uint16_t>& r) {
  if constexpr (HIDE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a = r.a[i];
      asm volatile("" : "+v"(a));
      r.a[i] = a;
    }
  }
}

// A lane's place for vector v of a row of L elements.  Every lane loads eight
// elements without a branch: the row's last, partial vector is read as the
// row's last eight elements, of which the first `drop` belong to the vector
// before; a vector past the row reads the same and drops them all.  Elements
// i < drop are left out of sums and stores.  SHORT: L < 8, one vector.
struct Place {
  int off, drop;
};
template <bool SHORT>
__device__ __forceinline__ Place place_of(int v, int L) {
  Place p;
  p.off = SHORT ? 0 : min(8 * v, L - 8);
  p.drop = SHORT ? (v == 0 ? 0 : 8) : min(8 * v - p.off, 8);
  return p;
}
template <bool SHORT, typename T>
__device__ __forceinline__ Row8<T> row_load(const T* row, Place pl, int L) {
  Row8<T> r;
  if constexpr (SHORT)
    r.load_short(row, L);
  else
    r.load(row + pl.off);
  return r;
}
template <bool SHORT, typename T>
__device__ __forceinline__ void row_store(T* row, Place pl, int L, const float* f) {
  if (!SHORT && pl.drop == 0) {
    Row8<T>::store(row + pl.off, f);
  } else {
    const int n = SHORT ? L : 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= pl.drop && i < n) Row8<T>::store1(row + pl.off + i, f[i]);
  }
}

// out[j] = sum over the nparts rows of part (nparts, n), j < n; columns
// [0, na) go to a, the rest to b.  Fixed order: no atomics, so the same inputs
// give the same bits.
hipError_t sum_parts(const float* part, int nparts, int n, float* a, int na, float* b,
                     hipStream_t st);

}  // namespace ssd
