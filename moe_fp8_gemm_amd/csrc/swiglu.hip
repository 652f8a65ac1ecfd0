// Gated activation between the two products of a layer: the next product's operand in 8 bits,
// an 8-bit checkpoint of its input for the backward pass, and its gradient.
//
// Mathematics.  h = [g | u], a = g s u with s = 1 / (1 + e^-g), everything in fp32 from
// the stored h, cast with the rules of the casts (NaN shows in the scale).  The checkpoint is the
// FP8 cast of h itself, in blocks of 128 that do not straddle the halves.  Gradient, at the stored h
// or at the values that the checkpoint stands for:
//   dg = da u s (1 + g (1 - s)),   du = da g s.
// e^-g is the hardware's 2^x of a rounded product: its relative error is |g| 2^-24 and a few
// units of the last place, far below a code or a 16-bit result.
//
// Bound by memory: each element is read once and written once, in 16-byte pieces (8 bytes of
// codes).  A layout's rows without a token are skipped: m_indices marks them row by row,
// masked_m ends a group's rows early.
#include "cast_rules.h"
#include "elem_types.h"
#include "layer_internal.h"

namespace dgfp8 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}
// g s: a gate of -1e30 gives 0, not -1e30 * 0 of an underflow in the wrong place
__device__ __forceinline__ float silu(float g) { return g * sigmoid(g); }

// Eight E4M3 codes times their scale.
__device__ __forceinline__ void widen_codes(u32x2 v, float s, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], true);
    x[4 * i] = lo[0] * s;
    x[4 * i + 1] = lo[1] * s;
    x[4 * i + 2] = hi[0] * s;
    x[4 * i + 3] = hi[1] * s;
  }
}

// Rows of a group that hold something.
__device__ __forceinline__ int64_t rows_in(const RowSet& at, int64_t g) {
  if (!at.masked_m) return at.group_rows;
  const int64_t n = at.masked_m[g];
  return n < 0 ? 0 : n > at.group_rows ? at.group_rows : n;
}

// Pieces of eight columns of a group's rows, in order, shared by the gridDim.x workgroups of
// group blockIdx.y: f(row, first column).  `per_row` pieces are a row.
template <class F>
__device__ __forceinline__ void each_piece(const RowSet& at, int64_t per_row, F&& f) {
  const int64_t g = blockIdx.y;
  const int64_t pieces = rows_in(at, g) * per_row;
  for (int64_t b = (int64_t)blockIdx.x * kThreads; b < pieces; b += (int64_t)gridDim.x * kThreads) {
    const int64_t row0 = b / per_row;
    const uint32_t in = (uint32_t)(b - row0 * per_row) + threadIdx.x;
    const uint32_t down = in / (uint32_t)per_row;
    const int64_t r = g * at.group_rows + row0 + down;
    if (b + threadIdx.x < pieces && (!at.m_indices || at.m_indices[r] >= 0))
      f(r, (int64_t)(in - down * (uint32_t)per_row) * 8);
  }
}

__device__ __forceinline__ void put_codes(uint8_t* q, float* sf, int64_t s0, int64_t s1, int64_t r, int64_t c, u32x2 code,
                                          float s) {
  __builtin_nontemporal_store(code, (u32x2*)(q + c));
  if ((threadIdx.x & 15) == 0) sf[r * s0 + (c >> 7) * s1] = s;
}

// inner is a multiple of 128, so a row is a multiple of 16 pieces and the 16 lanes of a
// block are in the same row.
template <class T, bool kKeep>
__global__ void __launch_bounds__(kThreads) swiglu_fp8_kernel(SwigluParams p) {
  typedef typename T::store E;
  each_piece(p.at, p.inner / 8, [&](int64_t r, int64_t c) {
    const E* h = (const E*)p.h + r * p.ldh + c;
    float g[8], u[8], a[8], s;
    widen_eight(stream_eight<T>(h), g);
    widen_eight(stream_eight<T>(h + p.inner), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = silu(g[i]) * u[i];
    const u32x2 code = fp8_of_block(a, p.ue8m0, s);
    put_codes(p.q + r * p.ldq, p.sf, p.sf_s0, p.sf_s1, r, c, code, s);
    if constexpr (kKeep) {
      const u32x2 cg = fp8_of_block(g, p.ue8m0, s);
      put_codes(p.hq + r * p.ldhq, p.hsf, p.hsf_s0, p.hsf_s1, r, c, cg, s);
      const u32x2 cu = fp8_of_block(u, p.ue8m0, s);
      put_codes(p.hq + r * p.ldhq, p.hsf, p.hsf_s0, p.hsf_s1, r, c + p.inner, cu, s);
    }
  });
}

// A workgroup a row (of its group): the row's maximum is needed before the first code, so its
// results stay in registers, up to kHeld x 2048.
template <class T, int kHeld>
__global__ void __launch_bounds__(kThreads) swiglu_int8_kernel(SwigluParams p) {
  typedef typename T::store E;
  const int64_t rows = rows_in(p.at, blockIdx.y);
  __shared__ uint32_t wave_max[2][kThreads / 64];
  int turn = 0;
  for (int64_t i0 = blockIdx.x; i0 < rows; i0 += gridDim.x) {
    const int64_t r = blockIdx.y * p.at.group_rows + i0;
    if (p.at.m_indices && p.at.m_indices[r] < 0) continue;   // the same for the whole workgroup
    const E* h = (const E*)p.h + r * p.ldh;
    float a[kHeld][8];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kThreads + threadIdx.x) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) a[i][j] = 0.0f;
      if (c >= p.inner) continue;
      float g[8], u[8];
      widen_eight(stream_eight<T>(h + c), g);
      widen_eight(stream_eight<T>(h + p.inner + c), u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[i][j] = silu(g[j]) * u[j];
        amax = max(amax, magnitude(a[i][j]));
      }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off, 64));
    // two buffers in turn: a row's maxima are read before those of the row after the next are written
    if ((threadIdx.x & 63) == 0) wave_max[turn][threadIdx.x >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) amax = max(amax, wave_max[turn][w]);
    turn ^= 1;
    const float s = int8_scale(amax);
    const Divisor d{s, 1.0f / s};
    if (threadIdx.x == 0) p.sf[r * p.sf_s0] = s;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kThreads + threadIdx.x) * 8;
      if (c < p.inner) *(u32x2*)(p.q + r * p.ldq + c) = int8_of_eight(a[i], d);
    }
  }
}

template <class T, bool kCodes, bool kCast>
__global__ void __launch_bounds__(kThreads) swiglu_grad_kernel(SwigluGradParams p) {
  typedef typename T::store E;
  each_piece(p.at, p.inner / 8, [&](int64_t r, int64_t c) {
    float d[8], g[8], u[8];
    if constexpr (kCodes) {
      const uint8_t* q = p.hq + r * p.ldhq + c;
      const float* sf = p.hsf + r * p.hsf_s0;
      const u32x2 qg = __builtin_nontemporal_load((const u32x2*)q);
      const u32x2 qu = __builtin_nontemporal_load((const u32x2*)(q + p.inner));
      const float sg = sf[(c >> 7) * p.hsf_s1], su = sf[((c + p.inner) >> 7) * p.hsf_s1];
      widen_codes(qg, sg, g);
      widen_codes(qu, su, u);
    } else {
      const E* h = (const E*)p.h + r * p.ldh + c;
      widen_eight(stream_eight<T>(h), g);
      widen_eight(stream_eight<T>(h + p.inner), u);
    }
    widen_eight(stream_eight<T>((const E*)p.da + r * p.ldda + c), d);
    float dg[8], du[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(g[i]);
      const float gs = g[i] * s;
      du[i] = d[i] * gs;
      dg[i] = d[i] * u[i] * __builtin_fmaf(gs, 1.0f - s, s);
    }
    E* dh = (E*)p.dh + r * p.lddh + c;
    store_eight<T>(dh, dg);
    store_eight<T>(dh + p.inner, du);
    if constexpr (kCast) {
      float s;
      const u32x2 cg = fp8_of_block(dg, p.ue8m0, s);
      put_codes(p.q + r * p.ldq, p.sf, p.sf_s0, p.sf_s1, r, c, cg, s);
      const u32x2 cu = fp8_of_block(du, p.ue8m0, s);
      put_codes(p.q + r * p.ldq, p.sf, p.sf_s0, p.sf_s1, r, c + p.inner, cu, s);
    }
  });
}

// Workgroups a group gets: all its pieces at once, less where there are many groups, whose
// rows are mostly few.
dim3 grid_of(const RowSet& at, int64_t items, int64_t per_block) {
  int64_t x = (items + per_block - 1) / per_block;
  const int64_t most = at.groups > 1 ? (4096 + at.groups - 1) / at.groups : (int64_t)1 << 22;
  if (x > most) x = most;
  return dim3((unsigned)x, (unsigned)at.groups);
}

template <class T>
hipError_t swiglu_fp8(const SwigluParams& p, hipStream_t stream) {
  const dim3 grid = grid_of(p.at, p.at.group_rows * (p.inner / 8), kThreads);
  if (p.hq) hipLaunchKernelGGL((swiglu_fp8_kernel<T, true>), grid, dim3(kThreads), 0, stream, p);
  else hipLaunchKernelGGL((swiglu_fp8_kernel<T, false>), grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <class T>
hipError_t swiglu_int8(const SwigluParams& p, hipStream_t stream) {
  const dim3 grid = grid_of(p.at, p.at.group_rows, 1), block(kThreads);
  constexpr int64_t kPass = kThreads * 8;
  if (p.inner <= kPass) hipLaunchKernelGGL((swiglu_int8_kernel<T, 1>), grid, block, 0, stream, p);
  else if (p.inner <= 2 * kPass) hipLaunchKernelGGL((swiglu_int8_kernel<T, 2>), grid, block, 0, stream, p);
  else if (p.inner <= 4 * kPass) hipLaunchKernelGGL((swiglu_int8_kernel<T, 4>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((swiglu_int8_kernel<T, 8>), grid, block, 0, stream, p);
  return hipGetLastError();
}

template <class T>
hipError_t swiglu_grad(const SwigluGradParams& p, hipStream_t stream) {
  const dim3 grid = grid_of(p.at, p.at.group_rows * (p.inner / 8), kThreads), block(kThreads);
  if (p.hq) {
    if (p.q) hipLaunchKernelGGL((swiglu_grad_kernel<T, true, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((swiglu_grad_kernel<T, true, false>), grid, block, 0, stream, p);
  } else {
    if (p.q) hipLaunchKernelGGL((swiglu_grad_kernel<T, false, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((swiglu_grad_kernel<T, false, false>), grid, block, 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu_fp8(const SwigluParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case DG_F32: return swiglu_fp8<F32>(p, stream);
    case DG_BF16: return swiglu_fp8<BF16>(p, stream);
    case DG_F16: return swiglu_fp8<F16>(p, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_swiglu_int8(const SwigluParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case DG_F32: return swiglu_int8<F32>(p, stream);
    case DG_BF16: return swiglu_int8<BF16>(p, stream);
    case DG_F16: return swiglu_int8<F16>(p, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_swiglu_grad(const SwigluGradParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case DG_F32: return swiglu_grad<F32>(p, stream);
    case DG_BF16: return swiglu_grad<BF16>(p, stream);
    case DG_F16: return swiglu_grad<F16>(p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace dgfp8
