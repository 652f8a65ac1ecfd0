// Host side of the mixture-of-experts entry points: argument checks (returned as
// status codes, before anything is launched) and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_util.h"
#include "moe_internal.h"

namespace dgfp8 {
namespace {

// A workgroup per token: keeps grid x block inside 32 bits.
constexpr int64_t kMaxTokens = (int64_t)1 << 23;
constexpr int64_t kMaxSlots = (int64_t)1 << 30;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

// Checks of the two routing calls, besides their own pointers.
dg_status check_route(int dtype, int64_t ld, int64_t ldi, int64_t ldw, int64_t tokens, int experts, int topk,
                      int score) {
  if (dtype != DG_F32 && dtype != DG_BF16 && dtype != DG_F16) return DG_ERROR_INVALID_VALUE;
  if (score != DG_ROUTE_SOFTMAX && score != DG_ROUTE_SIGMOID) return DG_ERROR_INVALID_VALUE;
  if (tokens < 0 || experts < 1 || topk < 1 || topk > experts) return DG_ERROR_INVALID_VALUE;
  if (ld < experts || ldi < topk || ldw < topk) return DG_ERROR_INVALID_VALUE;
  if (experts > kMaxExperts || topk > kMaxTopk || tokens > kMaxTokens) return DG_ERROR_NOT_SUPPORTED;
  if (!strides_ok({ld, ldi, ldw})) return DG_ERROR_NOT_SUPPORTED;
  return DG_SUCCESS;
}

// Checks of the row movers (dispatch, combination): a [tokens, topk] map into rows.
dg_status check_map(const void* slot_row, int64_t lds, int64_t tokens, int topk, int64_t rows) {
  if (tokens < 0 || rows < 0 || topk < 1) return DG_ERROR_INVALID_VALUE;
  if (tokens > 0 && (!slot_row || lds < topk)) return DG_ERROR_INVALID_VALUE;
  if (topk > kMaxTopk || tokens > kMaxTokens || rows > kMaxRows || !strides_ok({lds})) return DG_ERROR_NOT_SUPPORTED;
  if (!aligned(slot_row, 4)) return DG_ERROR_NOT_SUPPORTED;
  return DG_SUCCESS;
}

bool layout_sizes_ok(int64_t tokens, int topk, int experts) {
  return tokens >= 0 && topk >= 1 && topk <= kMaxTopk && experts >= 1 && experts <= kMaxExperts &&
         tokens <= kMaxSlots / topk;
}

dg_status layout(const int32_t* indices, int64_t ldi, int64_t tokens, int topk, int experts, int64_t max_m,
                 int64_t rows, int32_t* m_indices, int32_t* row_slot, int32_t* slot_row, int32_t* counts, void* ws,
                 size_t ws_bytes, void* stream) {
  if (tokens > 0 && (!indices || !slot_row || ldi < topk)) return DG_ERROR_INVALID_VALUE;
  if (!counts || (rows > 0 && !row_slot)) return DG_ERROR_INVALID_VALUE;
  if (!strides_ok({ldi}) || rows > kMaxRows) return DG_ERROR_NOT_SUPPORTED;
  if (!aligned(indices, 4) || !aligned(m_indices, 4) || !aligned(row_slot, 4) || !aligned(slot_row, 4) ||
      !aligned(counts, 4) || !aligned(ws, 16))
    return DG_ERROR_NOT_SUPPORTED;
  const size_t need =
      tokens * topk <= kOneLaunchSlots ? 0 : dg_expert_layout_workspace_size(tokens, topk, experts);
  if (need > 0 && (!ws || ws_bytes < need)) return DG_ERROR_INVALID_VALUE;
  LayoutParams p{};
  p.indices = indices; p.ldi = ldi;
  p.slots = tokens * topk; p.topk = topk; p.experts = experts;
  p.max_m = max_m; p.rows = rows;
  p.m_indices = m_indices; p.row_slot = row_slot; p.slot_row = slot_row; p.counts = counts;
  p.hist = static_cast<int32_t*>(ws);
  p.blocks = p.slots > 0 ? (int)ceil_div(p.slots, layout_block_slots(p.slots)) : 1;
  return of(launch_layout(p, static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace dgfp8

using namespace dgfp8;

DG_EXPORT dg_status dg_route_topk(const void* logits, int dtype, int64_t ld, const float* bias, int32_t* indices,
                                  int64_t ldi, float* weights, int64_t ldw, int64_t tokens, int experts, int topk,
                                  int groups, int topk_groups, int group_top2, int score, int renormalize,
                                  float scale, void* stream) {
  dg_status st = check_route(dtype, ld, ldi, ldw, tokens, experts, topk, score);
  if (st != DG_SUCCESS) return st;
  if (groups < 1 || topk_groups < 1 || topk_groups > groups || experts % groups != 0) return DG_ERROR_INVALID_VALUE;
  if (groups > kMaxExpertGroups) return DG_ERROR_NOT_SUPPORTED;
  if (tokens == 0) return DG_SUCCESS;
  if (!logits || !indices || !weights) return DG_ERROR_INVALID_VALUE;
  if (!aligned(logits, elem_bytes(dtype)) || !aligned(bias, 4) || !aligned(indices, 4) || !aligned(weights, 4))
    return DG_ERROR_NOT_SUPPORTED;
  RouteParams p{logits, ld, bias, indices, ldi, weights, ldw, tokens, experts, topk, groups, topk_groups, score,
                group_top2 ? 1 : 0, renormalize ? 1 : 0, scale};
  return of(launch_route(p, dtype, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_route_topk_grad(const void* logits, int dtype, int64_t ld, const int32_t* indices, int64_t ldi,
                                       const float* dweights, int64_t ldw, void* dlogits, int64_t ldd, int64_t tokens,
                                       int experts, int topk, int score, int renormalize, float scale,
                                       void* stream) {
  dg_status st = check_route(dtype, ld, ldi, ldw, tokens, experts, topk, score);
  if (st != DG_SUCCESS) return st;
  if (ldd < experts) return DG_ERROR_INVALID_VALUE;
  if (!strides_ok({ldd})) return DG_ERROR_NOT_SUPPORTED;
  if (tokens == 0) return DG_SUCCESS;
  if (!logits || !indices || !dweights || !dlogits) return DG_ERROR_INVALID_VALUE;
  if (!aligned(logits, elem_bytes(dtype)) || !aligned(dlogits, elem_bytes(dtype)) || !aligned(indices, 4) ||
      !aligned(dweights, 4))
    return DG_ERROR_NOT_SUPPORTED;
  RouteGradParams p{logits, ld, indices, ldi, dweights, ldw, dlogits, ldd, tokens, experts, topk, score,
                    renormalize ? 1 : 0, scale};
  return of(launch_route_grad(p, dtype, static_cast<hipStream_t>(stream)));
}

DG_EXPORT int64_t dg_expert_layout_rows(int64_t tokens, int topk, int experts) {
  if (!layout_sizes_ok(tokens, topk, experts)) return 0;
  const int64_t slots = tokens * topk;
  const int64_t used = slots < experts ? slots : experts;   // experts that can hold a slot
  return (slots + used * (kExpertAlignment - 1)) / kExpertAlignment * kExpertAlignment;
}

DG_EXPORT size_t dg_expert_layout_workspace_size(int64_t tokens, int topk, int experts) {
  if (!layout_sizes_ok(tokens, topk, experts)) return 0;
  const int64_t blocks = ceil_div(tokens * topk, layout_block_slots(tokens * topk));
  return blocks > 1 ? (size_t)layout_hist_rows(blocks) * experts * sizeof(int32_t) : 0;
}

DG_EXPORT dg_status dg_expert_layout_contiguous(const int32_t* indices, int64_t ldi, int64_t tokens, int topk,
                                                int experts, int64_t rows, int32_t* m_indices, int32_t* row_slot,
                                                int32_t* slot_row, int32_t* counts, void* ws, size_t ws_bytes,
                                                void* stream) {
  if (tokens < 0 || topk < 1 || experts < 1 || rows < 0) return DG_ERROR_INVALID_VALUE;
  if (!layout_sizes_ok(tokens, topk, experts)) return DG_ERROR_NOT_SUPPORTED;
  if (rows % kExpertAlignment != 0) return DG_ERROR_MISALIGNED_LAYOUT;
  if (rows > 0 && !m_indices) return DG_ERROR_INVALID_VALUE;
  return layout(indices, ldi, tokens, topk, experts, 0, rows, m_indices, row_slot, slot_row, counts, ws, ws_bytes,
                stream);
}

DG_EXPORT dg_status dg_expert_layout_masked(const int32_t* indices, int64_t ldi, int64_t tokens, int topk, int experts,
                                            int64_t max_m, int32_t* masked_m, int32_t* row_slot, int32_t* slot_row,
                                            void* ws, size_t ws_bytes, void* stream) {
  if (tokens < 0 || topk < 1 || experts < 1 || max_m < 1) return DG_ERROR_INVALID_VALUE;
  if (!layout_sizes_ok(tokens, topk, experts) || max_m > kMaxRows / experts) return DG_ERROR_NOT_SUPPORTED;
  return layout(indices, ldi, tokens, topk, experts, max_m, experts * max_m, nullptr, row_slot, slot_row, masked_m,
                ws, ws_bytes, stream);
}

DG_EXPORT dg_status dg_dispatch_cast_fp8(const void* x, int dtype, int64_t ldx, const int32_t* slot_row, int64_t lds,
                                         void* q, int64_t ldq, float* sf, int64_t sf_sm, int64_t sf_sk,
                                         int64_t tokens, int topk, int64_t rows, int64_t k, int ue8m0,
                                         void* stream) {
  if (dtype != DG_F32 && dtype != DG_BF16) return DG_ERROR_INVALID_VALUE;
  if (k < 0 || sf_sm < 0 || sf_sk < 0) return DG_ERROR_INVALID_VALUE;
  dg_status st = check_map(slot_row, lds, tokens, topk, rows);
  if (st != DG_SUCCESS || tokens == 0 || rows == 0 || k == 0) return st;
  if ((st = check_rows(x, ldx, k, elem_bytes(dtype))) != DG_SUCCESS) return st;
  if ((st = check_rows(q, ldq, k, 1)) != DG_SUCCESS) return st;
  if (!sf) return DG_ERROR_INVALID_VALUE;
  if (k % 128 != 0 || !aligned(sf, 4) || !strides_ok({sf_sm, sf_sk})) return DG_ERROR_NOT_SUPPORTED;
  if (k > (int64_t)1 << 24) return DG_ERROR_NOT_SUPPORTED;   // grid height
  DispatchParams p{x, ldx, slot_row, lds, topk, tokens, rows, k, static_cast<uint8_t*>(q), ldq, sf, sf_sm, sf_sk,
                   ue8m0 ? 1 : 0};
  return of(launch_dispatch_fp8(p, dtype, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_dispatch_cast_int8(const void* x, int dtype, int64_t ldx, const int32_t* slot_row, int64_t lds,
                                          void* q, int64_t ldq, float* sf, int64_t sf_s, int64_t tokens, int topk,
                                          int64_t rows, int64_t k, void* stream) {
  if (dtype != DG_F32 && dtype != DG_BF16) return DG_ERROR_INVALID_VALUE;
  if (k < 0 || sf_s < 0) return DG_ERROR_INVALID_VALUE;
  dg_status st = check_map(slot_row, lds, tokens, topk, rows);
  if (st != DG_SUCCESS || tokens == 0 || rows == 0 || k == 0) return st;
  if ((st = check_rows(x, ldx, k, elem_bytes(dtype))) != DG_SUCCESS) return st;
  if ((st = check_rows(q, ldq, k, 1)) != DG_SUCCESS) return st;
  if (!sf) return DG_ERROR_INVALID_VALUE;
  if (k % 16 != 0 || !aligned(sf, 4) || !strides_ok({sf_s})) return DG_ERROR_NOT_SUPPORTED;
  DispatchParams p{x, ldx, slot_row, lds, topk, tokens, rows, k, static_cast<uint8_t*>(q), ldq, sf, sf_s, 0, 0};
  return of(launch_cast_int8(p, dtype, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_combine(const void* y, int64_t ldy, const int32_t* slot_row, int64_t lds, const float* weights,
                               int64_t ldw, void* out, int out_dtype, int64_t ldo, int64_t tokens, int topk,
                               int64_t rows, int64_t h, void* stream) {
  if (out_dtype != DG_F32 && out_dtype != DG_BF16) return DG_ERROR_INVALID_VALUE;
  if (h < 0) return DG_ERROR_INVALID_VALUE;
  dg_status st = check_map(slot_row, lds, tokens, topk, rows);
  if (st != DG_SUCCESS || tokens == 0 || h == 0) return st;
  if (weights && ldw < topk) return DG_ERROR_INVALID_VALUE;
  if (!aligned(weights, 4) || !strides_ok({ldw})) return DG_ERROR_NOT_SUPPORTED;
  if (rows > 0 && (st = check_rows(y, ldy, h, 2)) != DG_SUCCESS) return st;
  if ((st = check_rows(out, ldo, h, elem_bytes(out_dtype))) != DG_SUCCESS) return st;
  if (h % 8 != 0 || h > (int64_t)1 << 24) return DG_ERROR_NOT_SUPPORTED;
  CombineParams p{y, ldy, slot_row, lds, weights, ldw, out, ldo, tokens, rows, h, topk};
  return of(launch_combine(p, out_dtype, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_combine_grad(const void* dout, int64_t ldo, const void* y, int64_t ldy,
                                    const int32_t* slot_row, int64_t lds, const int32_t* row_slot,
                                    const float* weights, int64_t ldw, void* dy, int64_t lddy, float* dweights,
                                    int64_t lddw, int64_t tokens, int topk, int64_t rows, int64_t h, void* stream) {
  if (h < 0) return DG_ERROR_INVALID_VALUE;
  dg_status st = check_map(slot_row, lds, tokens, topk, rows);
  if (st != DG_SUCCESS) return st;
  if (tokens > 0 && (!weights || !dweights || ldw < topk || lddw < topk)) return DG_ERROR_INVALID_VALUE;
  if (!aligned(weights, 4) || !aligned(dweights, 4) || !strides_ok({ldw, lddw})) return DG_ERROR_NOT_SUPPORTED;
  if (h % 8 != 0 || h > (int64_t)1 << 24) return DG_ERROR_NOT_SUPPORTED;
  if (tokens > 0 && h > 0 && (st = check_rows(dout, ldo, h, 2)) != DG_SUCCESS) return st;
  if (rows > 0 && h > 0) {
    if ((st = check_rows(y, ldy, h, 2)) != DG_SUCCESS) return st;
    if ((st = check_rows(dy, lddy, h, 2)) != DG_SUCCESS) return st;
  }
  if (tokens == 0 && (rows == 0 || h == 0)) return DG_SUCCESS;
  // read for every row, also where h == 0 leaves nothing to clear
  if (rows > 0 && !row_slot) return DG_ERROR_INVALID_VALUE;
  if (!aligned(row_slot, 4)) return DG_ERROR_NOT_SUPPORTED;
  if (tokens + rows / 64 >= 2 * kMaxTokens) return DG_ERROR_NOT_SUPPORTED;   // grid
  CombineGradParams p{dout, ldo, y, ldy, slot_row, lds, row_slot, weights, ldw, dy, lddy, dweights, lddw,
                      tokens, rows, h, topk};
  return of(launch_combine_grad(p, static_cast<hipStream_t>(stream)));
}

DG_EXPORT dg_status dg_per_token_cast_int8(const void* x, int dtype, int64_t ldx, void* q, int64_t ldq, float* sf,
                                           int64_t sf_s, int64_t m, int64_t k, void* stream) {
  if (dtype != DG_F32 && dtype != DG_BF16) return DG_ERROR_INVALID_VALUE;
  if (m < 0 || k < 0 || sf_s < 0) return DG_ERROR_INVALID_VALUE;
  if (m == 0 || k == 0) return DG_SUCCESS;
  dg_status st = check_rows(x, ldx, k, elem_bytes(dtype));
  if (st != DG_SUCCESS || (st = check_rows(q, ldq, k, 1)) != DG_SUCCESS) return st;
  if (!sf) return DG_ERROR_INVALID_VALUE;
  if (k % 16 != 0 || m > kMaxTokens || !aligned(sf, 4) || !strides_ok({sf_s})) return DG_ERROR_NOT_SUPPORTED;
  DispatchParams p{x, ldx, nullptr, 0, 1, m, m, k, static_cast<uint8_t*>(q), ldq, sf, sf_s, 0, 0};
  return of(launch_cast_int8(p, dtype, static_cast<hipStream_t>(stream)));
}
