// Root-mean-square norm of rows with the residual's addition, its rows written as they are
// or quantized for the next product, and its gradient.
//
// Mathematics.  h = x + r in fp32, rounded once to x's type; from the rounded row
//   rho = (sum h^2 / k + eps)^-1/2,  y = h rho w,
// so that the gradient, which has the stored h, is that of what was computed.  The
// cast takes y in fp32: codes and scales are those of the casts (NaN shows in the
// scale).  y is (h w) rho: fp32 holds the product of 16-bit h and w, so that one rounding stands before the cast's
// division, where 16-bit factors often make quotients on a midpoint of two codes (8192 rows of 7168: 4148 of 59 M codes
// beside those of the exact values, 5426 with (h rho) w).  Gradient, with n = h rho and m = sum(w dy n) / k:
//   dx = dh + rho (w dy - n m),   dw = sum over rows of dy n.
//
// Bound by memory: each row is read once, held in registers between its sum of squares and its output, and
// written once, past L2 where nothing near reads it.  Measured, bf16: 32768 rows of 7168 with residual to FP8
// (1.65 GB) 283 us, 5.8 TB/s; one such row 3.9 us, of which a launch that does nothing has 3.6; gradient of 16384
// rows with dh (0.94 GB) 181 us, 5.2 TB/s; 4099 rows of 2048 24 us, of which the sum of the workgroups' shares of dw
// is about 5.  Rows in a run for each XCD's L2 296 us, stores through the caches 290.
#include "cast_rules.h"
#include "elem_types.h"
#include "layer_internal.h"

namespace dgfp8 {
namespace {

// Sum over the lanes of a row: a wave, or all waves of the workgroup (part: one float a
// wave, not in use before).
template <int kLanes>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if constexpr (kLanes > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kLanes / 64; ++i) v += part[i];
  }
  return v;
}
template <int kLanes>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  if constexpr (kLanes > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kLanes / 64; ++i) v = max(v, part[i]);
  }
  return v;
}

// Eight weights as fp32.
template <class T>
__device__ __forceinline__ void weights_of(const void* w, int f32, int64_t c, float (&out)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = 1.0f;
  } else if (f32) {
    widen_eight(load_eight<F32>((const float*)w + c), out);
  } else {
    widen_eight(load_eight<T>((const typename T::store*)w + c), out);
  }
}

constexpr int group_threads(int lanes) { return lanes > 256 ? lanes : 256; }

// kLanes lanes a row, eight columns each, kHeld times.
template <class T, int kOut, int kLanes, int kHeld>
__global__ void __launch_bounds__(group_threads(kLanes)) norm_kernel(NormParams p) {
  constexpr int kRows = group_threads(kLanes) / kLanes;
  const int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes;
  if (r >= p.rows) return;   // with one row a workgroup all its waves leave
  const int lane = threadIdx.x % kLanes;
  __shared__ float part[kLanes / 64];
  __shared__ uint32_t top[kLanes / 64];
  typedef typename T::store E;
  const E* x = (const E*)p.x + r * p.ldx;
  Eight<T> v[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int64_t c = (int64_t)(i * kLanes + lane) * 8;
    v[i] = c < p.k ? load_eight<T>(x + c) : zero_eight<T>();
  }
  if (p.residual) {
    const E* res = (const E*)p.residual + r * p.ldr;
    Eight<T> u[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kLanes + lane) * 8;
      u[i] = c < p.k ? load_eight<T>(res + c) : zero_eight<T>();
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      float a[8], b[8];
      widen_eight(v[i], a);
      widen_eight(u[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
      v[i] = narrow_eight<T>(a);
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    float a[8];
    widen_eight(v[i], a);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(a[j], a[j], sum);
  }
  if (p.h) {
    E* h = (E*)p.h + r * p.ldh;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kLanes + lane) * 8;
      if (c < p.k) stream_out<T>(h + c, v[i]);
    }
  }
  sum = row_sum<kLanes>(sum, part);
  const float rho = 1.0f / __builtin_sqrtf(sum / (float)p.k + p.eps);
  if (lane == 0 && p.rstd) p.rstd[r] = rho;
  float y[kHeld][8];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int64_t c = (int64_t)(i * kLanes + lane) * 8;
    if (c < p.k) {
      float w[8];
      weights_of<T>(p.weight, p.weight_f32, c, w);
      widen_eight(v[i], y[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * w[j] * rho;   // h w of 16-bit types is exact: one rounding
      if (p.y) store_eight<T>((E*)p.y + r * p.ldy + c, y[i]);
      if constexpr (kOut == kNormFp8) {
        float s;
        const u32x2 code = fp8_of_block(y[i], p.ue8m0, s);   // k is a multiple of 128: a block's lanes are here together
        __builtin_nontemporal_store(code, (u32x2*)(p.q + r * p.ldq + c));
        if ((lane & 15) == 0) p.sf[r * p.sf_s0 + (c >> 7) * p.sf_s1] = s;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] = 0.0f;
    }
  }
  if constexpr (kOut == kNormInt8) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, magnitude(y[i][j]));
    const float s = int8_scale(row_max<kLanes>(amax, top));
    const Divisor d{s, 1.0f / s};
    if (lane == 0) p.sf[r * p.sf_s0] = s;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kLanes + lane) * 8;
      if (c < p.k) *(u32x2*)(p.q + r * p.ldq + c) = int8_of_eight(y[i], d);
    }
  }
}

// A workgroup takes rows b, b + blocks, ... and keeps its share of dw in registers; rows
// differ by kRows where a wave holds a row, and the waves' shares are added in order.  kAhead: the loads of
// the next row are issued before this row's sum, so that memory is busy through both (16384 rows of 7168: 198 us
// without); beyond 8192 columns the registers do not hold two rows.
template <class T, int kLanes, int kHeld, bool kAhead>
__global__ void __launch_bounds__(group_threads(kLanes), sizeof(typename T::store) == 2 && kAhead ? 4 : 1) norm_grad_kernel(NormGradParams p) {
  constexpr int kRows = group_threads(kLanes) / kLanes;
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  __shared__ float part[2][kLanes / 64];
  typedef typename T::store E;
  struct Row {
    Eight<T> g[kHeld], v[kHeld];
    float rho;
  };
  auto load = [&](int64_t r, Row& row) {
    const E* dy = (const E*)p.dy + r * p.lddy;
    const E* h = (const E*)p.h + r * p.ldh;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kLanes + lane) * 8;
      const bool in = c < p.k;
      row.g[i] = in ? stream_eight<T>(dy + c) : zero_eight<T>();
      row.v[i] = in ? stream_eight<T>(h + c) : zero_eight<T>();
    }
    row.rho = p.rstd[r];
  };
  float dw[kHeld][8];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  int turn = 0;
  const int64_t apart = (int64_t)p.blocks * kRows;
  int64_t r = (int64_t)blockIdx.x * kRows + sub;
  Row now;
  if (r < p.rows) load(r, now);
  for (; r < p.rows; r += apart) {
    Eight<T> u[kHeld];   // for the end of this row
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kLanes + lane) * 8;
      u[i] = c < p.k && p.dh ? stream_eight<T>((const E*)p.dh + r * p.lddh + c) : zero_eight<T>();
    }
    Row next;
    if constexpr (kAhead) {
      if (r + apart < p.rows) load(r + apart, next);
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kLanes + lane) * 8;
      if (c >= p.k) continue;
      float a[8], b[8], w[8];
      widen_eight(now.g[i], a);
      widen_eight(now.v[i], b);
      weights_of<T>(p.weight, p.weight_f32, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = a[j] * (b[j] * now.rho);
        dw[i][j] += t;
        dot = __builtin_fmaf(w[j], t, dot);
      }
    }
    // two buffers in turn: the sum of a row is read before the row after the next is written
    const float m = row_sum<kLanes>(dot, part[turn]) / (float)p.k;
    turn ^= 1;
    E* dx = (E*)p.dx + r * p.lddx;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kLanes + lane) * 8;
      if (c >= p.k) continue;
      float a[8], b[8], w[8], e[8];
      widen_eight(now.g[i], a);
      widen_eight(now.v[i], b);
      widen_eight(u[i], e);
      weights_of<T>(p.weight, p.weight_f32, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = __builtin_fmaf(now.rho, w[j] * a[j] - b[j] * now.rho * m, e[j]);
      store_eight<T>(dx + c, e);
    }
    if constexpr (kAhead) {
      now = next;
    } else {
      if (r + apart < p.rows) load(r + apart, now);
    }
  }
  if (!p.partial) return;
  float* out = p.partial + (int64_t)blockIdx.x * p.k;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * kLanes + lane) * 8;
      if (c >= p.k) continue;
      *(u32x4*)(out + c) = (u32x4){__float_as_uint(dw[i][0]), __float_as_uint(dw[i][1]), __float_as_uint(dw[i][2]), __float_as_uint(dw[i][3])};
      *(u32x4*)(out + c + 4) = (u32x4){__float_as_uint(dw[i][4]), __float_as_uint(dw[i][5]), __float_as_uint(dw[i][6]), __float_as_uint(dw[i][7])};
    }
  } else {
    __shared__ float share[kRows][kLanes * kHeld * 8];
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) share[sub][(i * kLanes + lane) * 8 + j] = dw[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < p.k; c += group_threads(kLanes)) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < kRows; ++q) s += share[q][c];
      out[c] = s;
    }
  }
}

// dw[c] = sum of the workgroups' shares, in an order that their number alone gives: 16
// columns a workgroup, 64 lanes a column.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* partial, int64_t k, int blocks, float* dweight) {
  const int64_t c = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
  const int slice = threadIdx.x >> 4;
  float s = 0.0f;
  if (c < k)
#pragma unroll 8
    for (int b = slice; b < blocks; b += 64) s += partial[(int64_t)b * k + c];
  __shared__ float part[64][17];
  part[slice][threadIdx.x & 15] = s;
  __syncthreads();
  if (slice < 16) {
#pragma unroll
    for (int i = 16; i < 64; i += 16) s += part[slice + i][threadIdx.x & 15];
  }
  __syncthreads();
  part[slice][threadIdx.x & 15] = s;
  __syncthreads();
  if (slice == 0 && c < k) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][threadIdx.x];
    dweight[c] = s;
  }
}

template <class T, int kOut, int kLanes, int kHeld>
void norm_of(const NormParams& p, hipStream_t stream) {
  constexpr int kRows = group_threads(kLanes) / kLanes;
  hipLaunchKernelGGL((norm_kernel<T, kOut, kLanes, kHeld>), dim3((unsigned)((p.rows + kRows - 1) / kRows)),
                     dim3(group_threads(kLanes)), 0, stream, p);
}

// Lanes of a row.  Few leave more rows to a CU and no barrier between a row's loads and its stores; a wave's registers
// bound them.  bf16 with residual to FP8, 32768 rows, in us, and with the next larger number of lanes: k 512 22
// and 35 (64 and 256 lanes), 1024 45 and 56, 4096 160 and 170 (256 and 512), 7168 283 and 325 (256 and 1024);
// 2048 86 with 64 and with 256.  16 rows: 1024 3.9 with 64 lanes and 3.3 with 256, 4096 4.2 with 256 and 3.6 with
// 512, 7168 5.5 with 256 and 3.9 with 1024.
template <class T, int kOut>
hipError_t norm(const NormParams& p, hipStream_t stream) {
  // No more rows than CUs: as many lanes as a row has work for.
  const bool few = p.rows <= 256;
  if (p.k <= 512) norm_of<T, kOut, 64, 1>(p, stream);
  else if (p.k <= 1024 && !few) norm_of<T, kOut, 64, 2>(p, stream);
  else if (p.k <= 2048) norm_of<T, kOut, 256, 1>(p, stream);
  else if (p.k <= 4096 && !few) norm_of<T, kOut, 256, 2>(p, stream);
  else if (p.k <= 8192 && !few) norm_of<T, kOut, 256, 4>(p, stream);
  else if (p.k <= 8192) norm_of<T, kOut, 1024, 1>(p, stream);
  else norm_of<T, kOut, 1024, 2>(p, stream);
  return hipGetLastError();
}

template <class T>
hipError_t norm(const NormParams& p, int out, hipStream_t stream) {
  switch (out) {
    case kNormRows: return norm<T, kNormRows>(p, stream);
    case kNormFp8: return norm<T, kNormFp8>(p, stream);
    case kNormInt8: return norm<T, kNormInt8>(p, stream);
  }
  return hipErrorInvalidValue;
}

template <class T, int kLanes, int kHeld, bool kAhead = true>
void norm_grad_of(const NormGradParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((norm_grad_kernel<T, kLanes, kHeld, kAhead>), dim3((unsigned)p.blocks), dim3(group_threads(kLanes)), 0,
                     stream, p);
}

// bf16 with weights' gradient and dh, 32768 rows, in us, and with the next larger number of lanes: k 512 32 and 67,
// 1024 56 and 79, 2048 108 and 141, 4096 202 and 213, 7168 355 and 392; 16 rows 5 to 7 with either.
template <class T>
hipError_t norm_grad(const NormGradParams& p, hipStream_t stream) {
  if (p.rows == 0) {   // dweight is cleared below
  } else if (p.k <= 512) norm_grad_of<T, 64, 1>(p, stream);
  else if (p.k <= 1024) norm_grad_of<T, 64, 2>(p, stream);
  else if (p.k <= 2048) norm_grad_of<T, 256, 1>(p, stream);
  else if (p.k <= 4096) norm_grad_of<T, 256, 2>(p, stream);
  else if (p.k <= 8192) norm_grad_of<T, 512, 2>(p, stream);
  else norm_grad_of<T, 1024, 2, false>(p, stream);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.dweight) return err;
  hipLaunchKernelGGL(norm_weight_kernel, dim3((unsigned)((p.k + 15) / 16)), dim3(1024), 0, stream, p.partial, p.k,
                     p.blocks, p.dweight);
  return hipGetLastError();
}

}  // namespace

// As many as run at once, each with the same number of rows but for the last few.  Beyond 1024 columns, where a workgroup
// takes row by row, one has up to four rows before there are more than 256: their shares of dw are longer
// than a row (1000 rows of 2048: 13.1 us and 16.4 with one row each; of 4096 19.9 and 24.2).
int norm_grad_blocks(int64_t rows, int64_t k) {
  const int64_t at_once = k <= 1024 ? 4 : 1;   // rows that a workgroup takes together
  const int64_t need = (rows + at_once - 1) / at_once;
  const int64_t most = k <= 4096 ? 1024 : 512;
  int64_t turns = (need + most - 1) / most;
  const int64_t some = need / 256 < 4 ? need / 256 : 4;
  if (at_once == 1 && turns < some) turns = some;
  return (int)(need < 1 ? 1 : (need + turns - 1) / turns);
}

hipError_t launch_norm(const NormParams& p, int dtype, int out, hipStream_t stream) {
  switch (dtype) {
    case DG_F32: return norm<F32>(p, out, stream);
    case DG_BF16: return norm<BF16>(p, out, stream);
    case DG_F16: return norm<F16>(p, out, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_norm_grad(const NormGradParams& p, int dtype, hipStream_t stream) {
  switch (dtype) {
    case DG_F32: return norm_grad<F32>(p, stream);
    case DG_BF16: return norm_grad<BF16>(p, stream);
    case DG_F16: return norm_grad<F16>(p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace dgfp8
