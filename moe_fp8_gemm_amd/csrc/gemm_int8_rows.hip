// int8 GEMM for a few rows (single tokens): D = sa sb A . B^T, dense with M <= 8 or
// masked groups of few rows each.
//
// Mathematics as in Int8Cfg (gemm_core.h): exact int32 sums, then fp32(sum) * sa *
// sb, each rounded to fp32, and one rounding to D's type, so the bits are those of the
// tiled kernels.
//
// Bound by reading B once.  With so few rows nothing of B is used twice, so it goes from
// memory to the registers that the matrix instructions read, without LDS and
// without a barrier in the K loop: a workgroup owns 16 columns (of a group), each of its
// 8 waves every 8th 128-wide piece of K.  A wave issues the loads of up to kAhead
// pieces (a whole 128-byte line of each of 16 rows of B apiece) before it multiplies the
// first, and the waves add up their sums through LDS at the end.  A's rows come from
// L2, the same for all workgroups; they are what grows with M.
// Measured against the best tiled plan, operands in HBM (us): 4096x7168 M = 1: 8.5
// to 11.1, M = 8: 9.5 to 11.4, M = 16: 10.6 to 11.4; 7168x16384 M = 1: 29.6 to
// 29.8, M = 8: 32.6 to 29.1, M = 16: 37.6 to 29.1; 2112x7168 M = 8: 8.7 to 9.7; 1024x512 M = 1:
// 2.8 to 3.8.  Hence up to 8 rows, whatever K: at 16384 deep that loses 12% with all 8 of them, and
// at 7168 deep another 8 rows would still gain.  2, 4 or 16 waves along K and 2 or 8 pieces ahead
// came within 5% of this choice or behind it.  The masked rule and its figures stand
// at run_masked_int8; 32 rows of A at a time lost to 16 at every count up to 16 and
// to the 64-row tiles beyond.
#include "dgfp8_device.h"

namespace dgfp8 {
namespace {

constexpr int kWaves = 8;
constexpr int kAhead = 4;    // 128-wide pieces of K in flight for a wave

// Rows m0 .. m0 + 15 (those below m) in the 16 columns from n0; a_rows, b_rows, sfa, sfb
// and d_off are the group's.
__device__ void rows_pass(const GemmParams& p, i32x4* part, const uint8_t* a_rows, const uint8_t* b_rows,
                          const float* sfa, const float* sfb, int64_t d_off, int64_t m0, int64_t m, int64_t n0) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t n_row = n0 + r16 < p.n ? n0 + r16 : p.n - 1;   // idle columns redo the last one
  const uint8_t* b = b_rows + n_row * p.ldb + q * 16;
  const uint8_t* a = a_rows + (m0 + r16 < m ? m0 + r16 : m - 1) * p.lda + q * 16;
  i32x4 acc = {0, 0, 0, 0};

  // Lane (r16, q) holds bytes 16q .. 16q + 15 of each 64-wide half of a piece, of
  // row r16 of B and of A alike: each half is one 16x16x64 product.
  const int whole = (int)(p.k / 128);
  int s = wave;
  for (; s + (kAhead - 1) * kWaves < whole; s += kAhead * kWaves) {
    i32x4 bv[kAhead][2], av[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) bv[u][h] = *(const i32x4*)(b + (int64_t)(s + u * kWaves) * 128 + h * 64);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) av[u][h] = *(const i32x4*)(a + (int64_t)(s + u * kWaves) * 128 + h * 64);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[u][h], av[u][h], acc, 0, 0, 0);
  }
  // the rest of this wave's pieces, the last of which K may cut short
  {
    const int pieces = (int)((p.k + 127) / 128);
    i32x4 bv[kAhead][2], av[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k0 = (int64_t)(s + u * kWaves) * 128 + h * 64;
        const bool in = s + u * kWaves < pieces && k0 + q * 16 < p.k;   // K is a multiple of 16
        bv[u][h] = in ? *(const i32x4*)(b + k0) : (i32x4){0, 0, 0, 0};
        av[u][h] = in ? *(const i32x4*)(a + k0) : (i32x4){0, 0, 0, 0};
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[u][h], av[u][h], acc, 0, 0, 0);
  }

  // ---- sum over the waves; result lane (r16, q), register i: row r16, column 4q + i
  part[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) acc += part[w * 64 + lane];
  const int64_t row = m0 + r16, n = n0 + 4 * q;
  if (row >= m || n >= p.n) return;
  const float sa = sfa[row * p.sfa_sm];
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = (float)acc[i] * sa * sfb[(n + i < p.n ? n + i : n) * p.sfb_sn];
  const bool wide = p.d_wide && n + 4 <= p.n;
  const int64_t at = d_off + row * p.ldd + n;
  if (p.out_type == DG_F32) {
    float* dst = (float*)p.d + at;
    if (wide) {
      *(f32x4*)dst = (f32x4){x[0], x[1], x[2], x[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.n) dst[i] = x[i];
    }
  } else {
    uint16_t* dst = p.d + at;
    uint32_t v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = p.out_type == DG_BF16 ? pack_bf16x2(x[2 * i], x[2 * i + 1]) : pack_f16x2(x[2 * i], x[2 * i + 1]);
    if (wide) {
      *(uint64_t*)dst = (uint64_t)v[1] << 32 | v[0];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.n) dst[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
  }
}

__global__ void __launch_bounds__(kWaves * 64) rows_kernel(GemmParams p) {
  __shared__ i32x4 part[kWaves * 64];
  rows_pass(p, part, p.a, p.b, p.sfa, p.sfb, 0, 0, p.m, (int64_t)blockIdx.x * 16);
}

// Workgroup (x, g) goes through the rows of group g, 16 at a time; two workgroups fit a CU.
__global__ void __launch_bounds__(kWaves * 64, 4) rows_masked_kernel(GemmParams p) {
  __shared__ i32x4 part[kWaves * 64];
  const int g = blockIdx.y;
  const int64_t listed = p.masked_m[g], m = listed < p.m ? listed : p.m;
  for (int64_t m0 = 0; m0 < m; m0 += 16) {
    if (m0 > 0) __syncthreads();      // the last pass has read its sums
    rows_pass(p, part, p.a + g * p.a_gs, p.b + g * p.b_gs, p.sfa + g * p.sfa_gs, p.sfb + g * p.sfb_gs, g * p.d_gs, m0, m,
              (int64_t)blockIdx.x * 16);
  }
}

}  // namespace

hipError_t launch_gemm_int8_rows(const GemmParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(rows_kernel, dim3((unsigned)((p.n + 15) / 16)), dim3(kWaves * 64), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_gemm_int8_rows_masked(const GemmParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(rows_masked_kernel, dim3((unsigned)((p.n + 15) / 16), (unsigned)p.num_groups), dim3(kWaves * 64), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace dgfp8
