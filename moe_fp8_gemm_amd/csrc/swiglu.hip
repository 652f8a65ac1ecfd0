// Gated activation between the two products of a layer: the next product's operand in 8 bits,
// an 8-bit checkpoint of its input for the backward pass, and its gradient.
//
// Mathematics.  h = [g | u], a = g s u with s = 1 / (1 + e^-g), everything in fp32 from
// the stored h, cast with the rules of the casts (NaN shows in the scale).  The checkpoint is the
// FP8 cast of h itself, in blocks of 128 that do not straddle the halves.  Gradient, at the stored h
// or at the values that the checkpoint stands for:
//   dg = da u s (1 + g (1 - s)),   du = da g s.
// e^-g is the hardware's 2^x of the rounded product t = -g log2 e, times 1 + (-g - t ln 2) for what the rounding
// left out: g s is within 4 x 2^-24 of itself for gates from -10 on and within 7.2 x 2^-24 down to -87, where ln 2 in
// fp32, off by 0.05 x 2^-24 of itself, is taken 87 times.
//
// Bound by memory: each element is read once and written once, in 16-byte pieces (8 bytes of
// codes), past L2.  A layout's rows without a token are skipped: m_indices marks them row by row,
// masked_m ends a group's rows early.  Measured, bf16: 32768 tokens' rows of 2 x 2048 among 256 experts' padding, with
// the checkpoint (476 MB) 102 us, 4.7 TB/s; the gradient from the checkpoint with its cast (680 MB) 131 us, 5.2 TB/s;
// 16 x 256 rows with at most 32 tokens each 4.7 us, 333 rows' gradient 4.2, of which a launch that does nothing has 3.6.
//
// Tried: rows in a run for each XCD's L2 155 and 170 us; 16 elements a thread side by side 135 and 191; codes
// written through the caches 102 and 133; the sigmoid without what the rounding of g log2 e left out: 3 us less, twice as many
// codes beside the exact value's.
#include "cast_rules.h"
#include "elem_types.h"
#include "layer_internal.h"

namespace dgfp8 {
namespace {

constexpr int kThreads = 256;

// Beyond 88 the sigmoid is 1, or below fp32's normal numbers; a NaN comes back with the gate itself, which is a
// factor of everything below.
__device__ __forceinline__ float sigmoid(float g) {
  const float c = __builtin_amdgcn_fmed3f(g, -88.0f, 88.0f);
  const float t = c * -1.44269504088896341f;
  const float e = __builtin_amdgcn_exp2f(t);
  const float d = 1.0f + __builtin_fmaf(e, __builtin_fmaf(t, -0.693147180559945309f, -c), e);
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);   // within half a unit of the last place or little more
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

// The same where blocks of 128 columns are cast: a workgroup takes 16 rows of kAtOnce neighbouring blocks, so that what
// it writes are whole lines of codes and, where a block's scales lie beside each other along the rows, 64 bytes of
// them.  f(row, first column, columns that are left): kAtOnce pieces 128 apart, all of whose loads
// are issued before the first is used.
template <int kAtOnce, class F>
__device__ __forceinline__ void each_block(const RowSet& at, int64_t inner, F&& f) {
  const int64_t g = blockIdx.y, rows = rows_in(at, g);
  const int64_t across = (inner + 128 * kAtOnce - 1) / (128 * kAtOnce);
  const int64_t units = (rows + 15) / 16 * across;
  for (int64_t b = blockIdx.x; b < units; b += gridDim.x) {
    const int64_t set = b / across, in = set * 16 + (threadIdx.x >> 4), r = g * at.group_rows + in;
    const int64_t c = (b - set * across) * (128 * kAtOnce) + (threadIdx.x & 15) * 8;
    if (in < rows && (!at.m_indices || at.m_indices[r] >= 0)) f(r, c, inner - c);
  }
}

__device__ __forceinline__ void put_codes(uint8_t* q, u32x2 code) { __builtin_nontemporal_store(code, (u32x2*)q); }

// Scales of the blocks that a row's 16 lanes cast together, side by side: one lane each writes them, in one
// store.
struct ScaleOut {
  float* at;       // this lane's
  int64_t step;    // to the next block's
  __device__ __forceinline__ void put(int blocks, float s0, float s1, float s2) const {
    const int l = threadIdx.x & 15;
    if (l < blocks) *at = l == 0 ? s0 : l == 1 ? s1 : s2;
  }
};

template <class T, bool kKeep, int kAtOnce>
__global__ void __launch_bounds__(kThreads) swiglu_fp8_kernel(SwigluParams p) {
  typedef typename T::store E;
  each_block<kAtOnce>(p.at, p.inner, [&](int64_t r, int64_t c, int64_t left) {
    const E* h = (const E*)p.h + r * p.ldh + c;
    Eight<T> hg[kAtOnce], hu[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (i * 128 < left) {   // the same for the whole workgroup
        hg[i] = stream_eight<T>(h + i * 128);
        hu[i] = stream_eight<T>(h + p.inner + i * 128);
      }
    }
    const int l = threadIdx.x & 15;
    uint8_t* q = p.q + r * p.ldq + c;
    uint8_t* hq = kKeep ? p.hq + r * p.ldhq + c : nullptr;
    ScaleOut out{p.sf + r * p.sf_s0 + (c >> 7) * p.sf_s1, p.sf_s1};
    if (kKeep && l > 0) out = {p.hsf + r * p.hsf_s0 + ((c + (l > 1 ? p.inner : 0)) >> 7) * p.hsf_s1, p.hsf_s1};
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (i * 128 >= left) break;
      float g[8], u[8], a[8], sa, sg = 0.0f, su = 0.0f;
      widen_eight(hg[i], g);
      widen_eight(hu[i], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = silu(g[j]) * u[j];
      put_codes(q + i * 128, fp8_of_block(a, p.ue8m0, sa));
      if constexpr (kKeep) {
        put_codes(hq + i * 128, fp8_of_block(g, p.ue8m0, sg));
        put_codes(hq + p.inner + i * 128, fp8_of_block(u, p.ue8m0, su));
      }
      out.put(kKeep ? 3 : 1, sa, sg, su);
      out.at += out.step;
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

// Eight columns of both halves and of the gradient, as they are stored.
template <class T, bool kCodes>
struct GradIn {
  Eight<T> d;
  Eight<T> g, u;     // from h,
  u32x2 qg, qu;      // or from the checkpoint
  float sg, su;
};

template <class T, bool kCodes, bool kCast, int kAtOnce>
__global__ void __launch_bounds__(kThreads) swiglu_grad_kernel(SwigluGradParams p) {
  typedef typename T::store E;
  typedef GradIn<T, kCodes> In;
  auto load = [&](int64_t r, int64_t c, In& in) {
    in.d = stream_eight<T>((const E*)p.da + r * p.ldda + c);
    if constexpr (kCodes) {
      const uint8_t* q = p.hq + r * p.ldhq + c;
      const float* sf = p.hsf + r * p.hsf_s0;
      in.qg = __builtin_nontemporal_load((const u32x2*)q);
      in.qu = __builtin_nontemporal_load((const u32x2*)(q + p.inner));
      in.sg = sf[(c >> 7) * p.hsf_s1];
      in.su = sf[((c + p.inner) >> 7) * p.hsf_s1];
    } else {
      const E* h = (const E*)p.h + r * p.ldh + c;
      in.g = stream_eight<T>(h);
      in.u = stream_eight<T>(h + p.inner);
    }
  };
  auto finish = [&](E* dh, uint8_t* q, const ScaleOut& out, const In& in) {
    float d[8], g[8], u[8];
    widen_eight(in.d, d);
    if constexpr (kCodes) {
      widen_codes(in.qg, in.sg, g);
      widen_codes(in.qu, in.su, u);
    } else {
      widen_eight(in.g, g);
      widen_eight(in.u, u);
    }
    float dg[8], du[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid(g[i]);
      const float gs = g[i] * s;
      du[i] = d[i] * gs;
      dg[i] = d[i] * u[i] * __builtin_fmaf(gs, 1.0f - s, s);
    }
    store_eight<T>(dh, dg);
    store_eight<T>(dh + p.inner, du);
    if constexpr (kCast) {
      float sg, su;
      put_codes(q, fp8_of_block(dg, p.ue8m0, sg));
      put_codes(q + p.inner, fp8_of_block(du, p.ue8m0, su));
      out.put(2, sg, su, 0.0f);
    }
  };
  if constexpr (kCodes || kCast) {
    each_block<kAtOnce>(p.at, p.inner, [&](int64_t r, int64_t c, int64_t left) {
      In in[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (i * 128 < left) load(r, c + i * 128, in[i]);
      E* dh = (E*)p.dh + r * p.lddh + c;
      uint8_t* q = kCast ? p.q + r * p.ldq + c : nullptr;
      ScaleOut out{};
      if constexpr (kCast)
        out = {p.sf + r * p.sf_s0 + ((c + (threadIdx.x & 15 ? p.inner : 0)) >> 7) * p.sf_s1, p.sf_s1};
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (i * 128 >= left) break;
        finish(dh + i * 128, q + i * 128, out, in[i]);
        out.at += out.step;
      }
    });
  } else {
    each_piece(p.at, p.inner / 8, [&](int64_t r, int64_t c) {
      In in;
      load(r, c, in);
      finish((E*)p.dh + r * p.lddh + c, nullptr, {}, in);
    });
  }
}

// Workgroups a group gets: all its pieces at once, less where there are many groups, whose
// rows are mostly few.
dim3 grid_of(const RowSet& at, int64_t items, int64_t per_block) {
  int64_t x = (items + per_block - 1) / per_block;
  const int64_t most = at.groups > 1 ? (4096 + at.groups - 1) / at.groups : (int64_t)1 << 22;
  if (x > most) x = most;
  return dim3((unsigned)x, (unsigned)at.groups);
}

// Blocks of 128 columns that a workgroup takes at once, where there are workgroups enough: 32768 rows of 2 x 2048, with
// the checkpoint and its gradient: 1 110 and 136 us, 2 99 and 127, 4 98 and 139, 8 112 and 148.  The rule counts a
// layout's rows, as the host knows no others; where few of the masked layout's hold a token, one block would be better:
// 64 x 256 rows of 2 x 2048, 63, 1011 and 7173 of them with a token, gradient with its cast, 1 block 5.4, 9.4 and 37.4
// us, 2 7.3, 13.6 and 39.5.
constexpr int kMany = 2;
bool many_blocks(const RowSet& at, int64_t inner) { return at.group_rows * at.groups * inner >= (int64_t)1 << 24; }
dim3 block_grid(const RowSet& at, int64_t inner, int at_once) {
  return grid_of(at, (at.group_rows + 15) / 16 * ((inner + 128 * at_once - 1) / (128 * at_once)), 1);
}

template <class T, bool kKeep>
void swiglu_fp8_of(const SwigluParams& p, hipStream_t stream) {
  if (many_blocks(p.at, p.inner))
    hipLaunchKernelGGL((swiglu_fp8_kernel<T, kKeep, kMany>), block_grid(p.at, p.inner, kMany), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((swiglu_fp8_kernel<T, kKeep, 1>), block_grid(p.at, p.inner, 1), dim3(kThreads), 0, stream, p);
}

template <class T>
hipError_t swiglu_fp8(const SwigluParams& p, hipStream_t stream) {
  if (p.hq) swiglu_fp8_of<T, true>(p, stream);
  else swiglu_fp8_of<T, false>(p, stream);
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

template <class T, bool kCodes, bool kCast>
void swiglu_grad_of(const SwigluGradParams& p, hipStream_t stream) {
  if constexpr (!kCodes && !kCast) {
    hipLaunchKernelGGL((swiglu_grad_kernel<T, false, false, 1>), grid_of(p.at, p.at.group_rows * (p.inner / 8), kThreads),
                       dim3(kThreads), 0, stream, p);
  } else if (many_blocks(p.at, p.inner)) {
    hipLaunchKernelGGL((swiglu_grad_kernel<T, kCodes, kCast, kMany>), block_grid(p.at, p.inner, kMany), dim3(kThreads), 0,
                       stream, p);
  } else {
    hipLaunchKernelGGL((swiglu_grad_kernel<T, kCodes, kCast, 1>), block_grid(p.at, p.inner, 1), dim3(kThreads), 0, stream,
                       p);
  }
}

template <class T>
hipError_t swiglu_grad(const SwigluGradParams& p, hipStream_t stream) {
  if (p.hq && p.q) swiglu_grad_of<T, true, true>(p, stream);
  else if (p.hq) swiglu_grad_of<T, true, false>(p, stream);
  else if (p.q) swiglu_grad_of<T, false, true>(p, stream);
  else swiglu_grad_of<T, false, false>(p, stream);
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
