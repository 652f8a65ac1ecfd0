// Launch parameters of the mixture-of-experts operators (routing, expert
// layout, dispatch, combine), shared by the host API and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/dgfp8.h"

namespace dgfp8 {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 64;
constexpr int kMaxExpertGroups = 64;
constexpr int kExpertAlignment = 128;   // rows: the contiguous layout's segments

struct RouteParams {
  const void* logits;             // [tokens, experts], row stride ld
  int64_t ld;
  const float* bias;              // [experts] or null
  int32_t* indices;               // [tokens, topk], row stride ldi
  int64_t ldi;
  float* weights;                 // [tokens, topk], row stride ldw
  int64_t ldw;
  int64_t tokens;
  int experts, topk;
  int groups, topk_groups;
  int score;                      // dg_route_score
  int group_top2;                 // group score: largest key (0), or sum of the two largest scores + bias (1)
  int renormalize;
  float scale;
};

struct RouteGradParams {
  const void* logits;
  int64_t ld;
  const int32_t* indices;
  int64_t ldi;
  const float* dweights;
  int64_t ldw;
  void* dlogits;                  // [tokens, experts] of the logits' type, row stride ldd
  int64_t ldd;
  int64_t tokens;
  int experts, topk;
  int score;
  int renormalize;
  float scale;
};

// Expert layout (see dg_expert_layout_contiguous / _masked).
struct LayoutParams {
  const int32_t* indices;         // [tokens, topk], row stride ldi
  int64_t ldi;
  int64_t slots;                  // tokens * topk
  int topk, experts;
  int64_t max_m;                  // masked layout: rows of an expert; 0: contiguous layout
  int64_t rows;                   // rows of the layout
  int32_t* m_indices;             // [rows] (contiguous) or null
  int32_t* row_slot;              // [rows]
  int32_t* slot_row;              // [tokens, topk]
  int32_t* counts;                // [experts]
  int32_t* hist;                  // [blocks, experts] (summed: [blocks + 1, experts]): workspace of large calls
  int blocks;                     // workgroups that share the slots
};
// One launch lays out this many slots, without a workspace (see moe_layout.hip).
constexpr int64_t kOneLaunchSlots = 3 * 1024;
// Slots of one workgroup: 1024 each, so that the work spreads; past 64 workgroups
// 4096, so that the counts each of them adds up stay few.
constexpr int64_t layout_block_slots(int64_t slots) { return slots <= 65536 ? 1024 : 4096; }
// Past this many workgroups a launch of its own sums their counts, so that the work stays in
// proportion to the slots (256 experts, top 8, us, without and with it: 64 workgroups 16.8 and 17.9, 128
// 20.9 and 19.4, 512 58 and 43, 8192 (4 M tokens) 5148 and 488).
constexpr int64_t kSumBlocks = 96;
constexpr int64_t layout_hist_rows(int64_t blocks) { return blocks > kSumBlocks ? blocks + 1 : blocks; }

// Cast of token rows into expert rows, and the plain int8 cast (slot_row null: row t).
struct DispatchParams {
  const void* x;                  // [tokens, k], row stride ldx
  int64_t ldx;
  const int32_t* slot_row;        // [tokens, topk], row stride lds
  int64_t lds;
  int topk;
  int64_t tokens, rows, k;
  uint8_t* q;                     // [rows, k], row stride ldq
  int64_t ldq;
  float* sf;                      // FP8: [rows, k/128] at (sf_s0, sf_s1); int8: [rows] at sf_s0
  int64_t sf_s0, sf_s1;
  int ue8m0;
};

struct CombineParams {
  const void* y;                  // bf16 [rows, h], row stride ldy
  int64_t ldy;
  const int32_t* slot_row;        // [tokens, topk], row stride lds
  int64_t lds;
  const float* weights;           // [tokens, topk], row stride ldw; null: ones
  int64_t ldw;
  void* out;                      // bf16 or fp32 [tokens, h], row stride ldo
  int64_t ldo;
  int64_t tokens, rows, h;
  int topk;
};

struct CombineGradParams {
  const void* dout;               // bf16 [tokens, h], row stride ldo
  int64_t ldo;
  const void* y;                  // bf16 [rows, h], row stride ldy
  int64_t ldy;
  const int32_t* slot_row;        // [tokens, topk], row stride lds
  int64_t lds;
  const int32_t* row_slot;        // [rows]
  const float* weights;           // [tokens, topk], row stride ldw
  int64_t ldw;
  void* dy;                       // bf16 [rows, h], row stride lddy
  int64_t lddy;
  float* dweights;                // [tokens, topk], row stride lddw
  int64_t lddw;
  int64_t tokens, rows, h;
  int topk;
};

hipError_t launch_layout(const LayoutParams& p, hipStream_t stream);
hipError_t launch_dispatch_fp8(const DispatchParams& p, int dtype, hipStream_t stream);
hipError_t launch_cast_int8(const DispatchParams& p, int dtype, hipStream_t stream);
hipError_t launch_combine(const CombineParams& p, int out_dtype, hipStream_t stream);
hipError_t launch_combine_grad(const CombineGradParams& p, hipStream_t stream);

hipError_t launch_route(const RouteParams& p, int dtype, hipStream_t stream);
hipError_t launch_route_grad(const RouteGradParams& p, int dtype, hipStream_t stream);

}  // namespace dgfp8
