// Host side of the norm, the gated activation and the weights' gradients: argument checks
// (returned as status codes, before anything is launched) and launches on the caller's
// stream.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_util.h"
#include "layer_internal.h"

namespace dgfp8 {
namespace {

// A workgroup a row: grid x block inside 32 bits, for 256 lanes and for the norm's 1024.
constexpr int64_t kMaxRows = (int64_t)1 << 23;
constexpr int64_t kMaxWideRows = (int64_t)1 << 21;
constexpr int64_t kWide = 8192;                        // columns
constexpr int64_t kMaxInner = (int64_t)1 << 24;
constexpr int64_t kMaxInnerInt8 = 16384;               // a row's results in registers
constexpr int64_t kMaxLd = ((int64_t)1 << 24) - 1;     // weights' gradients: 32 rows inside 2^31 bytes

bool is_dtype(int dtype) { return dtype == DG_F32 || dtype == DG_BF16 || dtype == DG_F16; }

// A weight of x's type or fp32, read in 16-byte pieces.
dg_status check_weight(const void* w, int weight_dtype, int dtype) {
  if (!w) return DG_SUCCESS;
  if (weight_dtype != dtype && weight_dtype != DG_F32) return DG_ERROR_INVALID_VALUE;
  return aligned(w, 16) ? DG_SUCCESS : DG_ERROR_NOT_SUPPORTED;
}

dg_status check_norm(int dtype, int64_t rows, int64_t k) {
  if (!is_dtype(dtype) || rows < 0 || k < 0) return DG_ERROR_INVALID_VALUE;
  return DG_SUCCESS;
}
dg_status check_width(int64_t rows, int64_t k) {
  return k % 8 != 0 || k > kMaxNormWidth || rows > (k > kWide ? kMaxWideRows : kMaxRows) ? DG_ERROR_NOT_SUPPORTED
                                                                                         : DG_SUCCESS;
}

// Everything but the quantized output.  launch: whether there is anything to do.
dg_status norm_of(NormParams& p, int dtype, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                  const void* weight, int weight_dtype, float eps, void* h, int64_t ldh, void* y, int64_t ldy,
                  float* rstd, int64_t rows, int64_t k, bool& launch) {
  launch = false;
  dg_status st = check_norm(dtype, rows, k);
  if (st != DG_SUCCESS) return st;
  if (!(eps >= 0.0f) || std::isinf(eps)) return DG_ERROR_INVALID_VALUE;
  if (rows == 0 || k == 0) return DG_SUCCESS;
  const int64_t el = elem_bytes(dtype);
  if ((st = check_rows(x, ldx, k, el)) != DG_SUCCESS) return st;
  if (residual && (st = check_rows(residual, ldr, k, el)) != DG_SUCCESS) return st;
  if (h && (st = check_rows(h, ldh, k, el)) != DG_SUCCESS) return st;
  if (y && (st = check_rows(y, ldy, k, el)) != DG_SUCCESS) return st;
  if ((st = check_weight(weight, weight_dtype, dtype)) != DG_SUCCESS) return st;
  if (!aligned(rstd, 4)) return DG_ERROR_NOT_SUPPORTED;
  if ((st = check_width(rows, k)) != DG_SUCCESS) return st;
  p = NormParams{x, ldx, residual, ldr, weight, weight_dtype == DG_F32 ? 1 : 0, eps, h, ldh, y, ldy, rstd,
                 nullptr, 0, nullptr, 0, 0, rows, k, 0};
  launch = true;
  return DG_SUCCESS;
}

// Rows of a layout.
dg_status check_set(RowSet& at, const int32_t* m_indices, const int32_t* masked_m, int num_groups, int64_t rows) {
  if (m_indices && masked_m) return DG_ERROR_INVALID_VALUE;
  if (masked_m && (num_groups < 1 || rows % num_groups != 0)) return DG_ERROR_INVALID_VALUE;
  if (!aligned(m_indices, 4) || !aligned(masked_m, 4)) return DG_ERROR_NOT_SUPPORTED;
  if (masked_m && num_groups > kMaxGroups) return DG_ERROR_NOT_SUPPORTED;
  const int64_t groups = masked_m ? num_groups : 1;
  at = RowSet{m_indices, masked_m, groups, rows / groups};
  return DG_SUCCESS;
}

dg_status check_scales(const float* sf, int64_t s0, int64_t s1) {
  if (!sf || s0 < 0 || s1 < 0) return DG_ERROR_INVALID_VALUE;
  return aligned(sf, 4) && strides_ok({s0, s1}) ? DG_SUCCESS : DG_ERROR_NOT_SUPPORTED;
}

// Codes [rows, cols] and their scales.
dg_status check_codes(const void* q, int64_t ldq, int64_t cols, const float* sf, int64_t s0, int64_t s1) {
  const dg_status st = check_rows(q, ldq, cols, 1);
  return st != DG_SUCCESS ? st : check_scales(sf, s0, s1);
}

dg_status weight_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* sf, int64_t sf_sm,
                      int64_t sf_sk, void* dw, int out_dtype, int64_t lddw, int64_t dw_group_stride,
                      const int32_t* counts, int groups, int64_t max_m, int64_t alignment, int accumulate, int64_t rows,
                      int64_t n, int64_t k, void* ws, size_t ws_bytes, void* stream) {
  if (out_dtype != DG_F32 && out_dtype != DG_BF16) return DG_ERROR_INVALID_VALUE;
  if (rows < 0 || n < 0 || k < 0) return DG_ERROR_INVALID_VALUE;
  if (accumulate && out_dtype != DG_F32) return DG_ERROR_NOT_SUPPORTED;
  if (n == 0 || k == 0) return DG_SUCCESS;
  const int64_t el = elem_bytes(out_dtype);
  dg_status st = check_rows(dw, lddw, k, el);
  if (st != DG_SUCCESS) return st;
  if (groups > 1 && dw_group_stride < 0) return DG_ERROR_INVALID_VALUE;
  if (!strides_ok({dw_group_stride}) || (groups > 1 && dw_group_stride * el % 16 != 0)) return DG_ERROR_NOT_SUPPORTED;
  if (groups > 1 && dw_group_stride < k) return DG_ERROR_INVALID_VALUE;   // they would write each other's elements
  if (rows > 0) {
    if ((st = check_rows(dy, lddy, n, 2)) != DG_SUCCESS) return st;
    if ((st = check_rows(x, ldx, k, sf ? 1 : 2)) != DG_SUCCESS) return st;
    if (sf && (st = check_scales(sf, sf_sm, sf_sk)) != DG_SUCCESS) return st;
    if (lddy > kMaxLd || ldx > kMaxLd || (sf && sf_sm > kMaxLd)) return DG_ERROR_NOT_SUPPORTED;
  }
  if (n % 8 != 0 || k % (sf ? 128 : 8) != 0 || n > kMaxLd || k > kMaxLd) return DG_ERROR_NOT_SUPPORTED;
  if (rows >= (int64_t)1 << 31 || groups > kMaxGroups || !aligned(counts, 4)) return DG_ERROR_NOT_SUPPORTED;
  if (!aligned(ws, 16)) return DG_ERROR_NOT_SUPPORTED;
  // the kernel counts tiles, and a round of workgroups past the last, in int: 2^22 tiles, 256 GB of fp32, leave room
  if (ceil_div(n, 128) * ceil_div(k, 128) * groups > (int64_t)1 << 22) return DG_ERROR_NOT_SUPPORTED;
  int splits = weight_grad_splits(rows, n, k, groups);
  if (!ws || ws_bytes < (size_t)splits * groups * n * k * sizeof(float)) splits = 1;
  WeightGradParams p{static_cast<const uint16_t*>(dy), lddy, x, ldx, sf, sf_sm, sf_sk, dw, lddw, dw_group_stride,
                     counts, max_m, alignment, groups, rows, n, k, accumulate ? 1 : 0, splits,
                     static_cast<float*>(ws)};
  return of(launch_weight_grad(p, sf != nullptr, out_dtype, static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace dgfp8

using namespace dgfp8;

DG_EXPORT dg_status dg_rms_norm(const void* x, int dtype, int64_t ldx, const void* residual, int64_t ldr,
                                const void* weight, int weight_dtype, float eps, void* h, int64_t ldh, void* y,
                                int64_t ldy, float* rstd, int64_t rows, int64_t k, void* stream) {
  NormParams p{};
  bool launch;
  const dg_status st =
      norm_of(p, dtype, x, ldx, residual, ldr, weight, weight_dtype, eps, h, ldh, y, ldy, rstd, rows, k, launch);
  if (st != DG_SUCCESS || !launch) return st;
  if (!y) return DG_ERROR_INVALID_VALUE;
  return of(launch_norm(p, dtype, kNormRows, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_rms_norm_cast_fp8(const void* x, int dtype, int64_t ldx, const void* residual, int64_t ldr,
                                         const void* weight, int weight_dtype, float eps, void* h, int64_t ldh,
                                         void* y, int64_t ldy, float* rstd, void* q, int64_t ldq, float* sf,
                                         int64_t sf_sm, int64_t sf_sk, int64_t rows, int64_t k, int ue8m0,
                                         void* stream) {
  NormParams p{};
  bool launch;
  dg_status st =
      norm_of(p, dtype, x, ldx, residual, ldr, weight, weight_dtype, eps, h, ldh, y, ldy, rstd, rows, k, launch);
  if (st != DG_SUCCESS || !launch) return st;
  if ((st = check_codes(q, ldq, k, sf, sf_sm, sf_sk)) != DG_SUCCESS) return st;
  if (k % 128 != 0) return DG_ERROR_NOT_SUPPORTED;
  p.q = static_cast<uint8_t*>(q); p.ldq = ldq;
  p.sf = sf; p.sf_s0 = sf_sm; p.sf_s1 = sf_sk;
  p.ue8m0 = ue8m0 ? 1 : 0;
  return of(launch_norm(p, dtype, kNormFp8, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_rms_norm_cast_int8(const void* x, int dtype, int64_t ldx, const void* residual, int64_t ldr,
                                          const void* weight, int weight_dtype, float eps, void* h, int64_t ldh,
                                          void* y, int64_t ldy, float* rstd, void* q, int64_t ldq, float* sf,
                                          int64_t sf_s, int64_t rows, int64_t k, void* stream) {
  NormParams p{};
  bool launch;
  dg_status st =
      norm_of(p, dtype, x, ldx, residual, ldr, weight, weight_dtype, eps, h, ldh, y, ldy, rstd, rows, k, launch);
  if (st != DG_SUCCESS || !launch) return st;
  if ((st = check_codes(q, ldq, k, sf, sf_s, 0)) != DG_SUCCESS) return st;
  if (k % 16 != 0) return DG_ERROR_NOT_SUPPORTED;
  p.q = static_cast<uint8_t*>(q); p.ldq = ldq;
  p.sf = sf; p.sf_s0 = sf_s;
  return of(launch_norm(p, dtype, kNormInt8, static_cast<hipStream_t>(stream)));
}

DG_EXPORT size_t dg_rms_norm_grad_workspace_size(int64_t rows, int64_t k) {
  if (rows <= 0 || k <= 0 || check_width(rows, k) != DG_SUCCESS) return 0;
  return (size_t)norm_grad_blocks(rows, k) * k * sizeof(float);
}

DG_EXPORT dg_status dg_rms_norm_grad(const void* dy, int dtype, int64_t lddy, const void* h, int64_t ldh,
                                     const void* weight, int weight_dtype, const float* rstd, const void* dh,
                                     int64_t lddh, void* dx, int64_t lddx, float* dweight, int64_t rows, int64_t k,
                                     void* ws, size_t ws_bytes, void* stream) {
  dg_status st = check_norm(dtype, rows, k);
  if (st != DG_SUCCESS || k == 0 || (rows == 0 && !dweight)) return st;
  const int64_t el = elem_bytes(dtype);
  if (rows > 0) {
    if ((st = check_rows(dy, lddy, k, el)) != DG_SUCCESS) return st;
    if ((st = check_rows(h, ldh, k, el)) != DG_SUCCESS) return st;
    if (dh && (st = check_rows(dh, lddh, k, el)) != DG_SUCCESS) return st;
    if ((st = check_rows(dx, lddx, k, el)) != DG_SUCCESS) return st;
    if (!rstd) return DG_ERROR_INVALID_VALUE;
  }
  if ((st = check_weight(weight, weight_dtype, dtype)) != DG_SUCCESS) return st;
  if (!aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(ws, 16)) return DG_ERROR_NOT_SUPPORTED;
  if ((st = check_width(rows, k)) != DG_SUCCESS) return st;
  if (dweight && rows > 0 && (!ws || ws_bytes < dg_rms_norm_grad_workspace_size(rows, k))) return DG_ERROR_INVALID_VALUE;
  NormGradParams p{dy, lddy, h, ldh, weight, weight_dtype == DG_F32 ? 1 : 0, rstd, dh, lddh, dx, lddx, dweight,
                   dweight ? static_cast<float*>(ws) : nullptr, rows, k, rows > 0 ? norm_grad_blocks(rows, k) : 0};
  return of(launch_norm_grad(p, dtype, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_swiglu_cast_fp8(const void* h, int dtype, int64_t ldh, const int32_t* m_indices,
                                       const int32_t* masked_m, int num_groups, void* q, int64_t ldq, float* sf,
                                       int64_t sf_sm, int64_t sf_sk, void* hq, int64_t ldhq, float* hsf,
                                       int64_t hsf_sm, int64_t hsf_sk, int64_t rows, int64_t inner, int ue8m0,
                                       void* stream) {
  if (!is_dtype(dtype) || rows < 0 || inner < 0) return DG_ERROR_INVALID_VALUE;
  SwigluParams p{};
  dg_status st = check_set(p.at, m_indices, masked_m, num_groups, rows);
  if (st != DG_SUCCESS || rows == 0 || inner == 0) return st;
  if ((st = check_rows(h, ldh, 2 * inner, elem_bytes(dtype))) != DG_SUCCESS) return st;
  if ((st = check_codes(q, ldq, inner, sf, sf_sm, sf_sk)) != DG_SUCCESS) return st;
  if (hq && (st = check_codes(hq, ldhq, 2 * inner, hsf, hsf_sm, hsf_sk)) != DG_SUCCESS) return st;
  if (inner % 128 != 0 || inner > kMaxInner || rows > kMaxRows) return DG_ERROR_NOT_SUPPORTED;
  p.h = h; p.ldh = ldh; p.inner = inner;
  p.q = static_cast<uint8_t*>(q); p.ldq = ldq; p.sf = sf; p.sf_s0 = sf_sm; p.sf_s1 = sf_sk;
  p.hq = static_cast<uint8_t*>(hq); p.ldhq = ldhq; p.hsf = hsf; p.hsf_s0 = hsf_sm; p.hsf_s1 = hsf_sk;
  p.ue8m0 = ue8m0 ? 1 : 0;
  return of(launch_swiglu_fp8(p, dtype, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_swiglu_cast_int8(const void* h, int dtype, int64_t ldh, const int32_t* m_indices,
                                        const int32_t* masked_m, int num_groups, void* q, int64_t ldq, float* sf,
                                        int64_t sf_s, int64_t rows, int64_t inner, void* stream) {
  if (!is_dtype(dtype) || rows < 0 || inner < 0) return DG_ERROR_INVALID_VALUE;
  SwigluParams p{};
  dg_status st = check_set(p.at, m_indices, masked_m, num_groups, rows);
  if (st != DG_SUCCESS || rows == 0) return st;
  if (inner == 0) {   // rows without columns have a scale all the same
    if ((st = check_scales(sf, sf_s, 0)) != DG_SUCCESS) return st;
  } else {
    if ((st = check_rows(h, ldh, 2 * inner, elem_bytes(dtype))) != DG_SUCCESS) return st;
    if ((st = check_codes(q, ldq, inner, sf, sf_s, 0)) != DG_SUCCESS) return st;
  }
  if (inner % 16 != 0 || inner > kMaxInnerInt8 || rows > kMaxRows) return DG_ERROR_NOT_SUPPORTED;
  p.h = h; p.ldh = ldh; p.inner = inner;
  p.q = static_cast<uint8_t*>(q); p.ldq = ldq; p.sf = sf; p.sf_s0 = sf_s;
  return of(launch_swiglu_int8(p, dtype, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_swiglu_grad(const void* da, int dtype, int64_t ldda, const void* h, int64_t ldh,
                                   const void* hq, int64_t ldhq, const float* hsf, int64_t hsf_sm, int64_t hsf_sk,
                                   const int32_t* m_indices, const int32_t* masked_m, int num_groups, void* dh,
                                   int64_t lddh, void* q, int64_t ldq, float* sf, int64_t sf_sm, int64_t sf_sk,
                                   int64_t rows, int64_t inner, int ue8m0, void* stream) {
  if (!is_dtype(dtype) || rows < 0 || inner < 0) return DG_ERROR_INVALID_VALUE;
  if (h && hq) return DG_ERROR_INVALID_VALUE;
  SwigluGradParams p{};
  dg_status st = check_set(p.at, m_indices, masked_m, num_groups, rows);
  if (st != DG_SUCCESS || rows == 0 || inner == 0) return st;
  const int64_t el = elem_bytes(dtype);
  if ((st = check_rows(da, ldda, inner, el)) != DG_SUCCESS) return st;
  if ((st = check_rows(dh, lddh, 2 * inner, el)) != DG_SUCCESS) return st;
  if (hq) {
    if ((st = check_codes(hq, ldhq, 2 * inner, hsf, hsf_sm, hsf_sk)) != DG_SUCCESS) return st;
  } else if ((st = check_rows(h, ldh, 2 * inner, el)) != DG_SUCCESS) {
    return st;
  }
  if (q && (st = check_codes(q, ldq, 2 * inner, sf, sf_sm, sf_sk)) != DG_SUCCESS) return st;
  if (inner % (hq || q ? 128 : 8) != 0 || inner > kMaxInner || rows > kMaxRows) return DG_ERROR_NOT_SUPPORTED;
  p.da = da; p.ldda = ldda; p.h = h; p.ldh = ldh;
  p.hq = static_cast<const uint8_t*>(hq); p.ldhq = ldhq; p.hsf = hsf; p.hsf_s0 = hsf_sm; p.hsf_s1 = hsf_sk;
  p.inner = inner; p.dh = dh; p.lddh = lddh;
  p.q = static_cast<uint8_t*>(q); p.ldq = ldq; p.sf = sf; p.sf_s0 = sf_sm; p.sf_s1 = sf_sk;
  p.ue8m0 = ue8m0 ? 1 : 0;
  return of(launch_swiglu_grad(p, dtype, static_cast<hipStream_t>(stream)));
}

DG_EXPORT size_t dg_weight_grad_workspace_size(int64_t rows, int64_t n, int64_t k, int num_groups) {
  if (rows <= 0 || n <= 0 || k <= 0 || num_groups < 1 || num_groups > kMaxGroups || n > kMaxLd || k > kMaxLd) return 0;
  const int splits = weight_grad_splits(rows, n, k, num_groups);
  return splits > 1 ? (size_t)splits * num_groups * n * k * sizeof(float) : 0;
}

DG_EXPORT dg_status dg_weight_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* sf,
                                   int64_t sf_sm, int64_t sf_sk, void* dw, int out_dtype, int64_t lddw, int accumulate,
                                   int64_t rows, int64_t n, int64_t k, void* ws, size_t ws_bytes, void* stream) {
  return weight_grad(dy, lddy, x, ldx, sf, sf_sm, sf_sk, dw, out_dtype, lddw, 0, nullptr, 1, 0, 1, accumulate, rows,
                     n, k, ws, ws_bytes, stream);
}

DG_EXPORT dg_status dg_m_grouped_weight_grad_contiguous(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                                        const float* sf, int64_t sf_sm, int64_t sf_sk, void* dw,
                                                        int out_dtype, int64_t lddw, int64_t dw_group_stride,
                                                        const int32_t* counts, int num_groups, int64_t alignment,
                                                        int accumulate, int64_t rows, int64_t n, int64_t k, void* ws,
                                                        size_t ws_bytes, void* stream) {
  if (num_groups < 0 || alignment < 1) return DG_ERROR_INVALID_VALUE;
  if (num_groups == 0) return DG_SUCCESS;
  if (!counts) return DG_ERROR_INVALID_VALUE;
  if (alignment >= (int64_t)1 << 31) return DG_ERROR_NOT_SUPPORTED;
  return weight_grad(dy, lddy, x, ldx, sf, sf_sm, sf_sk, dw, out_dtype, lddw, dw_group_stride, counts, num_groups, 0,
                     alignment, accumulate, rows, n, k, ws, ws_bytes, stream);
}

DG_EXPORT dg_status dg_m_grouped_weight_grad_masked(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                                    const float* sf, int64_t sf_sm, int64_t sf_sk, void* dw,
                                                    int out_dtype, int64_t lddw, int64_t dw_group_stride,
                                                    const int32_t* masked_m, int num_groups, int64_t max_m,
                                                    int accumulate, int64_t n, int64_t k, void* ws, size_t ws_bytes,
                                                    void* stream) {
  if (num_groups < 0 || max_m < 0) return DG_ERROR_INVALID_VALUE;
  if (num_groups == 0) return DG_SUCCESS;
  if (!masked_m) return DG_ERROR_INVALID_VALUE;
  if (num_groups > kMaxGroups || max_m >= ((int64_t)1 << 31) / num_groups) return DG_ERROR_NOT_SUPPORTED;
  // no rows at all: segments of no rows, one after the other
  return weight_grad(dy, lddy, x, ldx, sf, sf_sm, sf_sk, dw, out_dtype, lddw, dw_group_stride, masked_m, num_groups,
                     max_m, 1, accumulate, max_m * num_groups, n, k, ws, ws_bytes, stream);
}
