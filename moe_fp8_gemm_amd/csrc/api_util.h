// Small checks shared by the host entry points.
#pragma once

#include <cstdint>
#include <initializer_list>

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

}  // namespace dgfp8
