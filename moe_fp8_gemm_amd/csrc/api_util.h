// Small checks shared by the host entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/dgfp8.h"

#define DG_EXPORT extern "C" __attribute__((visibility("default")))

namespace dgfp8 {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Strides (elements) and sizes no real buffer comes near: 2^40.  Rejecting
// larger ones keeps every product of two of them inside int64 (on the host
// and in the kernels' 64-bit offset arithmetic).
constexpr int64_t kMaxStride = (int64_t)1 << 40;
inline bool strides_ok(std::initializer_list<int64_t> v) {
  for (int64_t x : v)
    if (x > kMaxStride) return false;
  return true;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline dg_status of(hipError_t err) { return err == hipSuccess ? DG_SUCCESS : DG_ERROR_LAUNCH; }

inline int64_t elem_bytes(int dtype) { return dtype == DG_F32 ? 4 : 2; }

// A matrix whose rows move in 16-byte pieces.
inline dg_status check_rows(const void* p, int64_t ld, int64_t cols, int64_t elem) {
  if (!p || ld < cols) return DG_ERROR_INVALID_VALUE;
  if (!strides_ok({ld, cols}) || !aligned(p, 16) || (ld * elem) % 16 != 0) return DG_ERROR_NOT_SUPPORTED;
  return DG_SUCCESS;
}

}  // namespace dgfp8
