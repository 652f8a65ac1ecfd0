// Launch parameters of the norm, the gated activation and the weights' gradients,
// shared by the host API and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/dgfp8.h"

namespace dgfp8 {

constexpr int kMaxNormWidth = 16384;   // columns of a row that a workgroup holds in registers
constexpr int kMaxGroups = 1024;

// What the normed rows become.
enum NormOut { kNormRows = 0, kNormFp8 = 1, kNormInt8 = 2 };

struct NormParams {
  const void* x;                  // [rows, k], row stride ldx
  int64_t ldx;
  const void* residual;           // [rows, k] of x's type, row stride ldr, or null
  int64_t ldr;
  const void* weight;             // [k], of x's type or fp32, or null: ones
  int weight_f32;
  float eps;
  void* h;                        // [rows, k] of x's type, row stride ldh, or null
  int64_t ldh;
  void* y;                        // [rows, k] of x's type, row stride ldy; null with a cast: none
  int64_t ldy;
  float* rstd;                    // [rows] or null
  uint8_t* q;                     // casts: [rows, k], row stride ldq
  int64_t ldq;
  float* sf;                      // FP8: [rows, k/128] at (sf_s0, sf_s1); int8: [rows] at sf_s0
  int64_t sf_s0, sf_s1;
  int64_t rows, k;
  int ue8m0;
};

struct NormGradParams {
  const void* dy;                 // [rows, k], row stride lddy
  int64_t lddy;
  const void* h;                  // [rows, k], row stride ldh
  int64_t ldh;
  const void* weight;             // as in NormParams
  int weight_f32;
  const float* rstd;              // [rows]
  const void* dh;                 // [rows, k], row stride lddh, or null
  int64_t lddh;
  void* dx;                       // [rows, k], row stride lddx
  int64_t lddx;
  float* dweight;                 // [k] or null
  float* partial;                 // [blocks, k]: workspace, null without dweight
  int64_t rows, k;
  int blocks;
};
// Workgroups that share the rows, each with its own partial sum of dweight.
int norm_grad_blocks(int64_t rows, int64_t k);

// Rows of a layout: all of them, those m_indices marks, or the first masked_m[g] of each
// group's.
struct RowSet {
  const int32_t* m_indices;       // [rows] or null
  const int32_t* masked_m;        // [groups] or null
  int64_t groups;                 // 1 without masked_m
  int64_t group_rows;             // rows / groups
};

struct SwigluParams {
  const void* h;                  // [rows, 2 * inner], row stride ldh
  int64_t ldh;
  RowSet at;
  int64_t inner;
  uint8_t* q;                     // [rows, inner], row stride ldq
  int64_t ldq;
  float* sf;                      // FP8: [rows, inner/128] at (sf_s0, sf_s1); int8: [rows] at sf_s0
  int64_t sf_s0, sf_s1;
  uint8_t* hq;                    // [rows, 2 * inner], row stride ldhq, or null: no checkpoint
  int64_t ldhq;
  float* hsf;                     // [rows, 2 * inner / 128] at (hsf_s0, hsf_s1)
  int64_t hsf_s0, hsf_s1;
  int ue8m0;
};

struct SwigluGradParams {
  const void* da;                 // [rows, inner], row stride ldda
  int64_t ldda;
  const void* h;                  // [rows, 2 * inner], row stride ldh, or null: from hq
  int64_t ldh;
  const uint8_t* hq;              // E4M3 [rows, 2 * inner], row stride ldhq
  int64_t ldhq;
  const float* hsf;               // [rows, 2 * inner / 128] at (hsf_s0, hsf_s1)
  int64_t hsf_s0, hsf_s1;
  RowSet at;
  int64_t inner;
  void* dh;                       // [rows, 2 * inner], row stride lddh
  int64_t lddh;
  uint8_t* q;                     // E4M3 [rows, 2 * inner], row stride ldq, or null: no cast
  int64_t ldq;
  float* sf;                      // [rows, 2 * inner / 128] at (sf_s0, sf_s1)
  int64_t sf_s0, sf_s1;
  int ue8m0;
};

struct WeightGradParams {
  const uint16_t* dy;             // bf16 [rows, n], row stride lddy
  int64_t lddy;
  const void* x;                  // bf16 or E4M3 [rows, k], row stride ldx (elements)
  int64_t ldx;
  const float* sf;                // E4M3: [rows, k/128] at (sf_s0, sf_s1)
  int64_t sf_s0, sf_s1;
  void* dw;                       // fp32 or bf16 [groups, n, k], row stride lddw, group stride dw_gs
  int64_t lddw, dw_gs;
  const int32_t* counts;          // [groups], or null: one group of all rows
  int64_t max_m;                  // masked layout: rows of a group's segment; 0: segments one after the other
  int64_t alignment;              //   each from a multiple of this many rows
  int groups;
  int64_t rows, n, k;
  int accumulate;                 // dw += (fp32 only)
  int splits;                     // workgroups that share a tile's rows
  float* partial;                 // [splits, groups, n, k] where splits > 1
  int past_l2;                    // the launch's own: how dW is written
};

hipError_t launch_norm(const NormParams& p, int dtype, int out, hipStream_t stream);
hipError_t launch_norm_grad(const NormGradParams& p, int dtype, hipStream_t stream);
hipError_t launch_swiglu_fp8(const SwigluParams& p, int dtype, hipStream_t stream);
hipError_t launch_swiglu_int8(const SwigluParams& p, int dtype, hipStream_t stream);
hipError_t launch_swiglu_grad(const SwigluGradParams& p, int dtype, hipStream_t stream);
hipError_t launch_weight_grad(const WeightGradParams& p, bool x_fp8, int out_dtype, hipStream_t stream);
int weight_grad_splits(int64_t rows, int64_t n, int64_t k, int groups);

}  // namespace dgfp8
