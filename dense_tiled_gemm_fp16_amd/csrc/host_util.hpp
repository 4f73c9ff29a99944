// Host helpers shared by the entry points' translation units: address spans,
// overlap tests and the device's compute-unit count.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/gemm_f16.h"

namespace gemmf16 {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Compute units of the current device, cached per device.
inline int device_cus(int* cus) {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return GEMM_ERR_HIP;
  if (dev >= 0 && dev < 64) {
    int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) {
      *cus = c;
      return GEMM_OK;
    }
  }
  int c = 0;
  if (hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || c <= 0)
    return GEMM_ERR_HIP;
  if (dev >= 0 && dev < 64) cache[dev].store(c, std::memory_order_relaxed);
  *cus = c;
  return GEMM_OK;
}

// Largest element offset of a rows x cols view, or false on int64 overflow.
inline bool view_span(int64_t rows, int64_t cols, int64_t sr, int64_t sc, int64_t* out) {
  int64_t a, b, s;
  if (__builtin_mul_overflow(rows - 1, sr, &a) || __builtin_mul_overflow(cols - 1, sc, &b) ||
      __builtin_add_overflow(a, b, &s) || s > INT64_MAX / 2 - 1)
    return false;
  *out = s;
  return true;
}

inline bool ranges_overlap(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) {
  return a0 < b1 && b0 < a1;
}

}  // namespace gemmf16
