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

// The same with the remainder's sign turned, which keeps the sign of a zero: q s - x of a zero x is +0, and
// q - 0 y has q's sign.
__device__ __forceinline__ float divide_signed(float x, Divisor d) {
#pragma clang fp contract(off)
  const float q = x * d.y;
  const float rem = __builtin_fmaf(q, d.s, -x);
  return __builtin_fmaf(-rem, d.y, q);
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
// block's scale: the same bits as fp8_scale and fp8_of_four in fewer instructions, where every block takes
// some thirty of them an element.  A NaN makes the scale a NaN (the maximum is the one that a NaN wins).  The
// quotient of the division by 448 is corrected as in divide(); an infinite or NaN maximum is the scale itself.
// No quotient exceeds 448 by more than its rounding (s is at least amax / 448 but for that), which the conversion
// rounds back to 448, so nothing is clamped; codes under an infinite or NaN scale are unspecified.
__device__ __forceinline__ u32x2 fp8_of_block(const float (&x)[8], int ue8m0, float& s) {
  float m = __builtin_elementwise_maximum(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
  for (int i = 2; i < 8; i += 2)
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(x[i])), fabsf(x[i + 1]));
  uint32_t amax = magnitude(m);
  // over the 16 lanes of a row of the wave, turned by 8, 4, 2 and 1: vector instructions, where shuffles go through LDS
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0x128, 0xF, 0xF, true));
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0x124, 0xF, 0xF, true));
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0x122, 0xF, 0xF, true));
  amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0x121, 0xF, 0xF, true));
  s = divide(fmaxf(__uint_as_float(amax), kAmaxFloor), {kE4M3Max, 1.0f / kE4M3Max});
  if (ue8m0) {
    uint32_t u = __float_as_uint(s);
    if (u & 0x007FFFFFu) u = (u & 0x7F800000u) + 0x00800000u;
    s = __uint_as_float(u);
  }
  if (amax >= 0x7F800000u) s = __uint_as_float(amax);
  const Divisor d{s, 1.0f / s};
  u32x2 code;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = divide_signed(x[4 * h + i], d);
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    code[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], v, true);
  }
  return code;
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
