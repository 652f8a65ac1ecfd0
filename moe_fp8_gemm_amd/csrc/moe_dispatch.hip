// Casts of token rows into the rows of their experts: FP8 with a scale for each
// 128-wide block, int8 with a scale for each row; and the int8 cast of plain rows.
//
// Mathematics.  FP8: per block amax = max |x|, s = max(amax, 1e-4) / 448 (rounded
// up to a power of two on request), q = E4M3(x / s): the rules of the per-token
// cast.  int8: per row s = max(amax, 1e-4) / 127, q = x / s rounded to the nearest
// whole number, ties to even.  Divisions are correctly rounded fp32.  A token's row
// is quantized once and written to the row of each of its experts.
//
// Bound by memory: tokens x k elements read, rows x k codes written.  Nothing is
// read twice, and the copies leave as whole 16-byte pieces, 1 KB a wave.
#include "cast_rules.h"
#include "elem_types.h"
#include "moe_internal.h"

namespace dgfp8 {
namespace {

constexpr int kThreads = 256;

// Token of a workgroup.  Workgroup b runs on XCD b % 8; a run of neighbouring
// tokens goes to each XCD, because neighbouring tokens fill neighbouring rows of an
// expert: where a block's scales lie beside each other along the rows, their 4-byte
// pieces then meet in one L2 before they leave, which the codes pass by without
// staying (non-temporal stores).  4096 tokens to 32768 rows of 7168, 297 MB: 64 us
// without either, 62 us with runs of tokens, 49 us (6.0 TB/s) with both.
__device__ __forceinline__ int64_t token_of(int64_t b, int64_t tokens) {
  const int64_t run = (tokens + 7) >> 3;
  return (b & 7) * run + (b >> 3);
}
int64_t token_grid(int64_t tokens) { return (tokens + 7) / 8 * 8; }

// Eight lanes own a 128-wide block, 16 elements each, so a wave covers eight
// blocks and a workgroup 4096 elements of one token.
template <class T>
__global__ void __launch_bounds__(kThreads) dispatch_fp8_kernel(DispatchParams p) {
  const int64_t t = token_of(blockIdx.x, p.tokens);
  const int64_t col = (int64_t)blockIdx.y * (kThreads * 16) + threadIdx.x * 16;
  if (t >= p.tokens || col >= p.k) return;   // k is a multiple of 128: a block's lanes leave together
  const typename T::store* src = (const typename T::store*)p.x + t * p.ldx + col;
  float x[16];
  {
    const Eight<T> a = load_eight<T>(src), b = load_eight<T>(src + 8);
    float lo[8], hi[8];
    widen_eight(a, lo);
    widen_eight(b, hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = lo[i];
      x[8 + i] = hi[i];
    }
  }
  float amax = 0.0f;   // a NaN does not count, as in the per-token cast
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 8));
  const float s = fp8_scale(__float_as_uint(amax), p.ue8m0);
  const Divisor d{s, 1.0f / s};
  u32x4 code;
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] = fp8_of_four(x + 4 * i, d);
  const int32_t* rows = p.slot_row + t * p.lds;
  const bool writes_scale = (threadIdx.x & 7) == 0;
  for (int j = 0; j < p.topk; ++j) {
    const int64_t r = rows[j];
    if (r < 0 || r >= p.rows) continue;
    __builtin_nontemporal_store(code, (u32x4*)(p.q + r * p.ldq + col));
    if (writes_scale) p.sf[r * p.sf_s0 + (col >> 7) * p.sf_s1] = s;
  }
}

// One workgroup per row.  The row's maximum is needed before the first code, so
// up to kHeld x 2048 elements stay in registers; what is beyond is read again.  Plain cast
// of bf16 rows, with the least kHeld that holds a row and with 4: 32768 x 2048 (201 MB)
// 42 us (4.8 TB/s) and 52, 4096 x 16384 40 and 49; 4096 x 7168 20.
template <class T, bool kScatter, int kHeld>
__global__ void __launch_bounds__(kThreads) cast_int8_kernel(DispatchParams p) {
  const int64_t t = blockIdx.x;
  const typename T::store* src = (const typename T::store*)p.x + t * p.ldx;
  constexpr int kPass = kThreads * 8;
  Eight<T> held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int64_t c = (int64_t)i * kPass + threadIdx.x * 8;
    held[i] = c < p.k ? load_eight<T>(src + c) : zero_eight<T>();
  }
  uint32_t amax = 0;
  auto take = [&](const Eight<T>& v) {
    float x[8];
    widen_eight(v, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, magnitude(x[i]));
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) take(held[i]);
  for (int64_t c = (int64_t)kHeld * kPass + threadIdx.x * 8; c < p.k; c += kPass) take(load_eight<T>(src + c));
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off, 64));
  __shared__ uint32_t wave_max[kThreads / 64];
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) amax = max(amax, wave_max[w]);
  const float s = int8_scale(amax);
  const Divisor d{s, 1.0f / s};
  auto code_of = [&](const Eight<T>& v) -> u32x2 {
    float x[8];
    widen_eight(v, x);
    return int8_of_eight(x, d);
  };
  const int copies = kScatter ? p.topk : 1;
  const int32_t* rows = kScatter ? p.slot_row + t * p.lds : nullptr;
  auto put = [&](int64_t c, u32x2 code) {
    for (int j = 0; j < copies; ++j) {
      const int64_t r = kScatter ? rows[j] : t;
      if (kScatter && (r < 0 || r >= p.rows)) continue;
      u32x2* dst = (u32x2*)(p.q + r * p.ldq + c);
      if constexpr (kScatter) {
        __builtin_nontemporal_store(code, dst);   // as in the FP8 dispatch
      } else {
        *dst = code;
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int64_t c = (int64_t)i * kPass + threadIdx.x * 8;
    if (c < p.k) put(c, code_of(held[i]));
  }
  for (int64_t c = (int64_t)kHeld * kPass + threadIdx.x * 8; c < p.k; c += kPass) put(c, code_of(load_eight<T>(src + c)));
  for (int j = threadIdx.x; j < copies; j += kThreads) {
    const int64_t r = kScatter ? rows[j] : t;
    if (!kScatter || (r >= 0 && r < p.rows)) p.sf[r * p.sf_s0] = s;
  }
}

template <class T, bool kScatter>
hipError_t cast_int8(const DispatchParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)p.tokens), block(kThreads);
  constexpr int64_t kPass = kThreads * 8;
  if (p.k <= kPass) {
    hipLaunchKernelGGL((cast_int8_kernel<T, kScatter, 1>), grid, block, 0, stream, p);
  } else if (p.k <= 2 * kPass) {
    hipLaunchKernelGGL((cast_int8_kernel<T, kScatter, 2>), grid, block, 0, stream, p);
  } else if (p.k <= 4 * kPass) {
    hipLaunchKernelGGL((cast_int8_kernel<T, kScatter, 4>), grid, block, 0, stream, p);
  } else {
    hipLaunchKernelGGL((cast_int8_kernel<T, kScatter, 8>), grid, block, 0, stream, p);
  }
  return hipGetLastError();
}

template <class T>
hipError_t dispatch_fp8(const DispatchParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)token_grid(p.tokens), (unsigned)((p.k + kThreads * 16 - 1) / (kThreads * 16)));
  hipLaunchKernelGGL((dispatch_fp8_kernel<T>), grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch_fp8(const DispatchParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case DG_F32: return dispatch_fp8<F32>(p, stream);
    case DG_BF16: return dispatch_fp8<BF16>(p, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_cast_int8(const DispatchParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case DG_F32: return p.slot_row ? cast_int8<F32, true>(p, stream) : cast_int8<F32, false>(p, stream);
    case DG_BF16: return p.slot_row ? cast_int8<BF16, true>(p, stream) : cast_int8<BF16, false>(p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace dgfp8
