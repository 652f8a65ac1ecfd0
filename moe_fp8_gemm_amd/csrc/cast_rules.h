// Scales and codes of the 8-bit casts, shared by the kernels that cast what they
// have just computed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "elem_types.h"

namespace dgfp8 {

constexpr float kE4M3Max = 448.0f;
constexpr float kInt8Max = 127.0f;
constexpr float kAmaxFloor = 1e-4f;

// |x| as bits: of the same order for whole numbers, and a NaN is the largest.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Correctly rounded fl32(x / s) for a normal positive s from y = fl32(1 / s): the
// quotient |x| y is within an ulp, its remainder is exact in one FMA and corrects
// it.  Quotients too small for that to hold are far below half a code.
struct Divisor {
  float s, y;
};
__device__ __forceinline__ float divide(float x, Divisor d) {
#pragma clang fp contract(off)
  const float q = x * d.y;
  const float rem = __builtin_fmaf(-q, d.s, x);
  return __builtin_fmaf(rem, d.y, q);
}

__device__ __forceinline__ float fp8_scale(uint32_t amax, int ue8m0) {
  float s = fmaxf(__uint_as_float(amax), kAmaxFloor) / kE4M3Max;
  if (ue8m0) {
    uint32_t u = __float_as_uint(s);
    if (u & 0x007FFFFFu) u = (u & 0x7F800000u) + 0x00800000u;
    s = __uint_as_float(u);
  }
  return s;
}

// As fp8_scale from a maximum in which a NaN counts (magnitude): such a block's scale
// is a NaN, which the products show.
__device__ __forceinline__ float fp8_scale_or_nan(uint32_t amax, int ue8m0) {
  return amax > 0x7F800000u ? __builtin_nanf("") : fp8_scale(amax, ue8m0);
}

__device__ __forceinline__ uint32_t fp8_of_four(const float* x, Divisor d) {
  float t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    t[i] = __builtin_copysignf(fminf(divide(fabsf(x[i]), d), kE4M3Max), x[i]);
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], v, true);
  return (uint32_t)v;
}

// Codes of eight elements of a 128-wide block that 16 neighbouring lanes hold, and the
// block's scale.
__device__ __forceinline__ u32x2 fp8_of_block(const float (&x)[8], int ue8m0, float& s) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, magnitude(x[i]));
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off, 16));
  s = fp8_scale_or_nan(amax, ue8m0);
  const Divisor d{s, 1.0f / s};
  return (u32x2){fp8_of_four(x, d), fp8_of_four(x + 4, d)};
}

// A row's int8 scale: a row with a NaN gets a NaN scale (and an infinite one an
// infinite scale), which the product's row shows.
__device__ __forceinline__ float int8_scale(uint32_t amax) {
  return amax > 0x7F800000u ? __builtin_nanf("") : fmaxf(__uint_as_float(amax), kAmaxFloor) / kInt8Max;
}

__device__ __forceinline__ u32x2 int8_of_eight(const float (&x)[8], Divisor d) {
  uint32_t whole[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(divide(x[i], d), -kInt8Max), kInt8Max);   // NaN -> -127: any finite code
    // at 1.5 * 2^23 fp32 holds whole numbers: the sum is q rounded to nearest even, its low
    // byte the code
    whole[i] = __float_as_uint(q + 0x1.8p23f);
  }
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(whole[4 * h + 1], whole[4 * h], 0x0C0C0400);
    const uint32_t hi = __builtin_amdgcn_perm(whole[4 * h + 3], whole[4 * h + 2], 0x0C0C0400);
    c[h] = __builtin_amdgcn_perm(hi, lo, 0x05040100);
  }
  return c;
}

}  // namespace dgfp8
