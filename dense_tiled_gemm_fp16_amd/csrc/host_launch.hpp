// Host helpers of the entry points that launch by kernel address: byte ranges
// of views, grids and the launch itself.
#pragma once

#include "host_util.hpp"

namespace gemmf16 {

struct Range {
  uintptr_t lo, hi;
};

// Byte range of rows x row_bytes bytes with row stride ld; false on overflow.
inline bool byte_rows(const void* p, int64_t rows, int64_t ld, int64_t row_bytes, Range* r) {
  int64_t a;
  if (__builtin_mul_overflow(rows - 1, ld, &a) || __builtin_add_overflow(a, row_bytes, &a) ||
      a > INT64_MAX / 2)
    return false;
  r->lo = (uintptr_t)p;
  r->hi = r->lo + (uintptr_t)a;
  return r->hi >= r->lo;
}

// Byte range of a rows x cols view with element strides; false on overflow.
inline bool byte_view(const void* p, int64_t rows, int64_t cols, int64_t sr, int64_t sc, int64_t elem, Range* r) {
  int64_t span;
  return view_span(rows, cols, sr, sc, &span) && span <= INT64_MAX / 16 && byte_rows(p, 1, 1, (span + 1) * elem, r);
}

// Whether the elements of a rows x cols view (whose range is known not to overflow)
// are apart from each other, as an output's have to be.
inline bool apart(int64_t rows, int64_t cols, int64_t sr, int64_t sc) {
  return rows == 1 || cols == 1 || sr > (cols - 1) * sc || sc > (rows - 1) * sr;
}

inline bool overlap(const Range& a, const Range& b) { return ranges_overlap(a.lo, a.hi, b.lo, b.hi); }

// A launch takes fewer than 2^32 work items along x.
inline bool fits_x(int64_t gx, int threads) { return gx < (INT64_C(1) << 32) / threads; }

// n workgroups (of up to 512) as a grid that a launch takes (rounded up).
inline dim3 wide_grid(int64_t n) {
  constexpr int64_t kX = INT64_C(1) << 22;
  return n <= kX ? dim3((unsigned)n) : dim3((unsigned)kX, (unsigned)cdiv(n, kX));
}
constexpr int64_t kMaxWide = INT64_C(65535) << 22;

inline int run(const void* fn, dim3 grid, int threads, void* args, hipStream_t s) {
  void* p[] = {args};
  return hipLaunchKernel(fn, grid, dim3((unsigned)threads), p, 0, s) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

// The last cache holds 256 MiB: what a call moves beyond half as much again need
// not stay in it for the next one.
constexpr double kOnceBytes = 384.0 * (1 << 20);

// A call's workspace: the caller's (checked), or allocated in stream order and
// given back in that order by done().
class Workspace {
 public:
  int take(void* given, size_t given_bytes, size_t need, hipStream_t s) {
    s_ = s;
    if (need == 0) return GEMM_OK;
    if (given) {
      if (given_bytes < need || ((uintptr_t)given & 255u)) return GEMM_ERR_WORKSPACE;
      p_ = given;
      return GEMM_OK;
    }
    if (hipMallocAsync(&p_, need, s) != hipSuccess) return GEMM_ERR_HIP;
    own_ = true;
    return GEMM_OK;
  }
  void* get() const { return p_; }
  int done(int rc) {
    if (own_ && hipFreeAsync(p_, s_) != hipSuccess && rc == GEMM_OK) rc = GEMM_ERR_HIP;
    own_ = false;
    return rc;
  }

 private:
  void* p_ = nullptr;
  hipStream_t s_ = nullptr;
  bool own_ = false;
};

}  // namespace gemmf16
