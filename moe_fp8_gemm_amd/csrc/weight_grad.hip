// Weights' gradients, grouped by expert with any number of rows: dW[e] = sum over the rows r
// of expert e of dy[r]^T x[r], x as 16-bit rows or as E4M3 codes with a scale for each 128 columns.
//
// Mathematics.  A product whose contraction runs over rows, the slow dimension of both operands.  dy and x
// enter the bf16 matrix instructions; a code times its scale is rounded to bf16 (not at all where the
// scale is a power of two, as with exponent-only scales: 4 significant bits stay).  Sums are
// fp32.  Rows behind an expert's last are read as zeros, whatever they hold.
//
// Staging.  64 rows of both operands go through registers into one of two LDS stages, as bf16 rows.
// ds_read_b64_tr_b16 turns a 4 x 16 piece of rows into the matrix instruction's
// fragments: each lane gets 4 rows of one column.  Both operands meet in the same order of
// rows, which is all that the contraction needs.  Rows are stored with their 32-byte units
// permuted by the row's number, so that the 8 rows that half a wave reads lie in 8 different
// bank groups.
#include "dgfp8_device.h"
#include "layer_internal.h"

namespace dgfp8 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 64;   // rows of a stage

// Segment of group g: first row and rows, inside [0, p.rows].
__device__ __forceinline__ void segment(const WeightGradParams& p, int g, int64_t& first, int64_t& count) {
  if (!p.counts) {
    first = 0;
    count = p.rows;
    return;
  }
  const int64_t mine = p.counts[g] < 0 ? 0 : p.counts[g];
  if (p.max_m > 0) {
    first = (int64_t)g * p.max_m;
    count = mine < p.max_m ? mine : p.max_m;
    return;
  }
  // the sum over the groups before, by every wave for itself
  int64_t before = 0;
  for (int i = threadIdx.x & 63; i < g; i += 64) {
    const int64_t c = p.counts[i] < 0 ? 0 : p.counts[i];
    before += (c + p.alignment - 1) / p.alignment * p.alignment;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) before += __shfl_xor(before, off, 64);
  before = (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(before >> 32)) << 32) |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)before));
  first = before < p.rows ? before : p.rows;
  count = mine < p.rows - first ? mine : p.rows - first;
}

// A descriptor over `rows` rows of `cols` elements, so that what lies behind reads as zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const void* base, int64_t first, int64_t rows, int64_t ld,
                                                          int64_t cols, int bytes) {
  const int64_t n = rows <= 0 ? 0 : rows < kStep ? rows : kStep;
  const int64_t len = n == 0 ? 0 : ((n - 1) * ld + cols) * bytes;
  return __builtin_amdgcn_make_buffer_rsrc((void*)((const char*)base + first * ld * bytes), 0, (int)len, kRawBufferFlags);
}

template <int kTn, int kTk, int kWavesN, int kWavesK, bool kFp8>
struct Shape {
  static constexpr int kThreads = kWavesN * kWavesK * 64;
  static constexpr int kPitchN = kTn * 2, kPitchK = kTk * 2;   // bytes of an LDS row
  static constexpr int kFragN = kTn / kWavesN / 16, kFragK = kTk / kWavesK / 16;
  static constexpr int kLoadsN = kStep * kTn * 2 / 16 / kThreads;              // 16-byte pieces a thread
  static constexpr int kLoadsK = kStep * kTk * (kFp8 ? 1 : 2) / 16 / kThreads;
};

// byte of 32-byte unit u of LDS row r
template <int kPitch>
__device__ __forceinline__ uint32_t unit_at(int r, int u) {
  return r * kPitch + ((u ^ (r & 7)) << 5);
}

template <int kTn, int kTk, int kWavesN, int kWavesK, bool kFp8, bool kF32>
__global__ void __launch_bounds__(kWavesN * kWavesK * 64, 2) weight_grad_kernel(WeightGradParams p) {
  typedef Shape<kTn, kTk, kWavesN, kWavesK, kFp8> S;
  __shared__ __attribute__((aligned(128))) uint8_t lds_n[2][kStep * S::kPitchN];
  __shared__ __attribute__((aligned(128))) uint8_t lds_k[2][kStep * S::kPitchK];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / kWavesK, wk = wave % kWavesK;
  const int tiles_n = (int)((p.n + kTn - 1) / kTn), tiles_k = (int)((p.k + kTk - 1) / kTk);
  // unit -> (group, split, tile); a run of neighbouring units for each XCD
  const int64_t units = (int64_t)p.groups * p.splits * tiles_n * tiles_k;
  const int64_t run = (units + 7) >> 3;
  int64_t unit = (int64_t)(blockIdx.x & 7) * run + (blockIdx.x >> 3);
  if (unit >= units) return;
  const int tk = (int)(unit % tiles_k);
  unit /= tiles_k;
  const int tn = (int)(unit % tiles_n);
  unit /= tiles_n;
  const int split = (int)(unit % p.splits), g = (int)(unit / p.splits);
  int64_t first, count;
  segment(p, g, first, count);
  const int64_t steps = (count + kStep - 1) / kStep;
  const int64_t share = (steps + p.splits - 1) / p.splits;
  const int64_t s0 = split * share < steps ? split * share : steps;
  const int64_t s1 = s0 + share < steps ? s0 + share : steps;
  const int64_t n0 = (int64_t)tn * kTn, k0 = (int64_t)tk * kTk;

  f32x4 acc[S::kFragN][S::kFragK];
#pragma unroll
  for (int i = 0; i < S::kFragN; ++i)
#pragma unroll
    for (int j = 0; j < S::kFragK; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};

  // this thread's pieces: 16 bytes of dy, 16 bytes of x
  u32x4 in_n[S::kLoadsN], in_k[S::kLoadsK];
  float sc[S::kLoadsK];
  constexpr int kPerN = kTn / 8;                        // pieces of a row
  constexpr int kPerK = kTk / (kFp8 ? 16 : 8);
  auto load = [&](int64_t s) {
    const int64_t row = s * kStep, left = count - row;
    const __amdgpu_buffer_rsrc_t rn = rows_at(p.dy + n0, first + row, left, p.lddy, p.n - n0, 2);
    const __amdgpu_buffer_rsrc_t rk = rows_at((const uint8_t*)p.x + k0 * (kFp8 ? 1 : 2), first + row, left, p.ldx,
                                              p.k - k0, kFp8 ? 1 : 2);
#pragma unroll
    for (int i = 0; i < S::kLoadsN; ++i) {
      const int piece = i * S::kThreads + threadIdx.x;
      in_n[i] = __builtin_amdgcn_raw_buffer_load_b128(rn, (int)((piece / kPerN) * p.lddy * 2 + (piece % kPerN) * 16), 0, 0);
    }
#pragma unroll
    for (int i = 0; i < S::kLoadsK; ++i) {
      const int piece = i * S::kThreads + threadIdx.x;
      const int r = piece / kPerK, c = piece % kPerK;
      in_k[i] = __builtin_amdgcn_raw_buffer_load_b128(rk, (int)(r * p.ldx * (kFp8 ? 1 : 2) + c * 16), 0, 0);
      if constexpr (kFp8) {
        const int64_t kb = (k0 + c * 16) >> 7;
        sc[i] = r < left && k0 + c * 16 < p.k ? p.sf[(first + row + r) * p.sf_s0 + kb * p.sf_s1] : 0.0f;
      }
    }
  };
  auto store = [&](int stage) {
#pragma unroll
    for (int i = 0; i < S::kLoadsN; ++i) {
      const int piece = i * S::kThreads + threadIdx.x;
      const int r = piece / kPerN, c = piece % kPerN;
      *(u32x4*)(lds_n[stage] + unit_at<S::kPitchN>(r, c >> 1) + (c & 1) * 16) = in_n[i];
    }
#pragma unroll
    for (int i = 0; i < S::kLoadsK; ++i) {
      const int piece = i * S::kThreads + threadIdx.x;
      const int r = piece / kPerK, c = piece % kPerK;
      if constexpr (kFp8) {
        u32x4 lo, hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)in_k[i][j], false);
          const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)in_k[i][j], true);
          const uint32_t w0 = pack_bf16x2(a[0] * sc[i], a[1] * sc[i]), w1 = pack_bf16x2(b[0] * sc[i], b[1] * sc[i]);
          if (j < 2) {
            lo[2 * j] = w0;
            lo[2 * j + 1] = w1;
          } else {
            hi[2 * j - 4] = w0;
            hi[2 * j - 3] = w1;
          }
        }
        uint8_t* dst = lds_k[stage] + unit_at<S::kPitchK>(r, c);
        *(u32x4*)dst = lo;
        *(u32x4*)(dst + 16) = hi;
      } else {
        *(u32x4*)(lds_k[stage] + unit_at<S::kPitchK>(r, c >> 1) + (c & 1) * 16) = in_k[i];
      }
    }
  };

  // Fragment of 16 columns (unit u) and rows 32 kk ..: this lane's column is u * 16 + lane % 16; its
  // rows are 4 (lane / 16) .. and 16 + 4 (lane / 16) .. .
  const int lrow = (lane >> 4) * 4 + ((lane & 15) >> 2);
  const uint32_t lbyte = (lane & 3) * 8;
  auto frag = [&](const uint8_t* stage, int pitch, int kk, int u) -> bf16x8 {
    const uint8_t* a = stage + (kk * 32 + lrow) * pitch + ((u ^ (lrow & 7)) << 5) + lbyte;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LAS s16x4*)(uint32_t)(uintptr_t)(DG_LAS const uint8_t*)a);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (DG_LAS s16x4*)(uint32_t)(uintptr_t)(DG_LAS const uint8_t*)(a + 16 * pitch));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  if (s0 < s1) {
    load(s0);
    store(0);
    __syncthreads();
  }
  for (int64_t s = s0; s < s1; ++s) {
    const int stage = (int)(s - s0) & 1;
    if (s + 1 < s1) load(s + 1);
#pragma unroll
    for (int kk = 0; kk < kStep / 32; ++kk) {
      bf16x8 fn[S::kFragN], fk[S::kFragK];
#pragma unroll
      for (int i = 0; i < S::kFragN; ++i) fn[i] = frag(lds_n[stage], S::kPitchN, kk, wn * S::kFragN + i);
#pragma unroll
      for (int j = 0; j < S::kFragK; ++j) fk[j] = frag(lds_k[stage], S::kPitchK, kk, wk * S::kFragK + j);
#pragma unroll
      for (int i = 0; i < S::kFragN; ++i)
#pragma unroll
        for (int j = 0; j < S::kFragK; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fk[j], fn[i], acc[i][j], 0, 0, 0);
    }
    if (s + 1 < s1) store(stage ^ 1);
    __syncthreads();
  }

  // lane: column n = lane % 16 of fragment i, rows k = 4 (lane / 16) .. of fragment j
  const int64_t gn = n0 + wn * S::kFragN * 16 + (lane & 15), gk = k0 + wk * S::kFragK * 16 + (lane >> 4) * 4;
#pragma unroll
  for (int i = 0; i < S::kFragN; ++i) {
    const int64_t n = gn + i * 16;
    if (n >= p.n) continue;
#pragma unroll
    for (int j = 0; j < S::kFragK; ++j) {
      const int64_t k = gk + j * 16;
      if (k >= p.k) continue;   // k is a multiple of 8: four columns are in or out together
      f32x4 v = acc[i][j];
      if (p.splits > 1) {
        *(f32x4*)(p.partial + (((int64_t)split * p.groups + g) * p.n + n) * p.k + k) = v;
      } else if constexpr (kF32) {
        f32x4* dst = (f32x4*)((float*)p.dw + g * p.dw_gs + n * p.lddw + k);
        if (p.accumulate) v += *dst;
        *dst = v;
      } else {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        *(u32x2*)((uint16_t*)p.dw + g * p.dw_gs + n * p.lddw + k) =
            (u32x2){pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
      }
    }
  }
}

// dW from the partial sums of the splits, in their order; four columns a thread.
template <bool kF32>
__global__ void __launch_bounds__(256) weight_grad_sum_kernel(WeightGradParams p) {
  const int64_t per = p.n * (p.k / 4), all = per * p.groups;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= all) return;
  const int64_t g = i / per, in = i - g * per, n = in / (p.k / 4), k = (in - n * (p.k / 4)) * 4;
  f32x4 v = *(const f32x4*)(p.partial + i * 4);
  for (int s = 1; s < p.splits; ++s) v += *(const f32x4*)(p.partial + (s * all + i) * 4);
  if constexpr (kF32) {
    f32x4* dst = (f32x4*)((float*)p.dw + g * p.dw_gs + n * p.lddw + k);
    if (p.accumulate) v += *dst;
    *dst = v;
  } else {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    *(u32x2*)((uint16_t*)p.dw + g * p.dw_gs + n * p.lddw + k) = (u32x2){pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
  }
}

int64_t tiles(int64_t n, int64_t k, int64_t tn, int64_t tk) { return ((n + tn - 1) / tn) * ((k + tk - 1) / tk); }

// 256 x 256 tiles need 256 of them to fill the device.
bool big_tiles(int64_t n, int64_t k, int groups) { return tiles(n, k, 256, 256) * groups >= 200; }

template <int kTn, int kTk, int kWavesN, int kWavesK>
hipError_t launch(const WeightGradParams& p, bool x_fp8, bool f32, hipStream_t stream) {
  const int64_t units = (int64_t)p.groups * p.splits * tiles(p.n, p.k, kTn, kTk);
  const dim3 grid((unsigned)((units + 7) / 8 * 8)), block(kWavesN * kWavesK * 64);
  if (x_fp8) {
    if (f32) hipLaunchKernelGGL((weight_grad_kernel<kTn, kTk, kWavesN, kWavesK, true, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((weight_grad_kernel<kTn, kTk, kWavesN, kWavesK, true, false>), grid, block, 0, stream, p);
  } else {
    if (f32) hipLaunchKernelGGL((weight_grad_kernel<kTn, kTk, kWavesN, kWavesK, false, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((weight_grad_kernel<kTn, kTk, kWavesN, kWavesK, false, false>), grid, block, 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace

int weight_grad_splits(int64_t rows, int64_t n, int64_t k, int groups) {
  if (big_tiles(n, k, groups)) return 1;
  const int64_t units = tiles(n, k, 128, 128) * groups;
  const int64_t steps = (rows / groups + kStep - 1) / kStep;   // of a group of average size
  int64_t s = units > 0 ? 512 / units : 1;
  if (s > steps / 4) s = steps / 4;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

hipError_t launch_weight_grad(const WeightGradParams& p, bool x_fp8, int out_dtype, hipStream_t stream) {
  const bool f32 = out_dtype == DG_F32;
  hipError_t err = big_tiles(p.n, p.k, p.groups) ? launch<256, 256, 2, 4>(p, x_fp8, f32, stream)
                                                 : launch<128, 128, 2, 2>(p, x_fp8, f32, stream);
  if (err != hipSuccess || p.splits <= 1) return err;
  const int64_t all = (int64_t)p.groups * p.n * (p.k / 4);
  const dim3 grid((unsigned)((all + 255) / 256));
  if (f32) hipLaunchKernelGGL((weight_grad_sum_kernel<true>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((weight_grad_sum_kernel<false>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dgfp8
