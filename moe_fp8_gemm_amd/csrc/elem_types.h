// Element types of the kernels that move rows, and their conversions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dgfp8 {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct F32 { typedef float store; };
struct BF16 { typedef uint16_t store; };
struct F16 { typedef uint16_t store; };

__device__ __forceinline__ float widen(F32, float v) { return v; }
__device__ __forceinline__ float widen(BF16, uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float widen(F16, uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
// One rounding to nearest even, where a result leaves fp32.
__device__ __forceinline__ float narrow(F32, float v) { return v; }
__device__ __forceinline__ uint16_t narrow(BF16, float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint16_t narrow(F16, float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

// Eight consecutive elements at a 16-byte boundary, as loaded: one register
// quad of 16-bit elements, two of fp32.
template <class T>
struct Eight {
  u32x4 q[sizeof(typename T::store) / 2];
};
template <class T>
__device__ __forceinline__ Eight<T> load_eight(const typename T::store* src) {
  Eight<T> v;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(typename T::store) / 2); ++i) v.q[i] = ((const u32x4*)src)[i];
  return v;
}
// The same for what is read once: passed through without being kept in L2.
template <class T>
__device__ __forceinline__ Eight<T> stream_eight(const typename T::store* src) {
  Eight<T> v;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(typename T::store) / 2); ++i)
    v.q[i] = __builtin_nontemporal_load((const u32x4*)src + i);
  return v;
}
template <class T>
__device__ __forceinline__ Eight<T> zero_eight() {
  Eight<T> v;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(typename T::store) / 2); ++i) v.q[i] = (u32x4){0, 0, 0, 0};
  return v;
}
template <class T>
__device__ __forceinline__ void widen_eight(const Eight<T>& v, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(typename T::store) == 4) {
      x[i] = __uint_as_float(v.q[i / 4][i % 4]);
    } else {
      x[i] = widen(T{}, (uint16_t)(v.q[0][i / 2] >> (16 * (i & 1))));
    }
  }
}
template <class T>
__device__ __forceinline__ Eight<T> narrow_eight(const float (&x)[8]) {
  Eight<T> v;
  if constexpr (sizeof(typename T::store) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.q[i / 4][i % 4] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v.q[0][i] = (uint32_t)narrow(T{}, x[2 * i]) | ((uint32_t)narrow(T{}, x[2 * i + 1]) << 16);
  }
  return v;
}
// Stores pass through as well: the rows moved here exceed L2 many times over.
template <class T>
__device__ __forceinline__ void stream_out(typename T::store* dst, const Eight<T>& v) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(typename T::store) / 2); ++i) __builtin_nontemporal_store(v.q[i], (u32x4*)dst + i);
}
template <class T>
__device__ __forceinline__ void store_eight(typename T::store* dst, const float (&x)[8]) {
  stream_out<T>(dst, narrow_eight<T>(x));
}

// LDS written by one lane and read by another lane of the same wave.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

}  // namespace dgfp8
