// Host side of include/gemm_mx4.h: argument validation and launches of the
// MX FP4 quantiser, its inverse and the products with MX4 weights.  Everything
// is checked before the first HIP call, so on any error nothing is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_mx4.h"
#include "host_util.hpp"
#include "mx4_convert.hpp"
#include "strip_kernel.hpp"

using namespace gemmf16;

namespace {

constexpr int64_t kMaxGrid = (INT64_C(1) << 31) - 1;

int64_t elem_size(int32_t fmt) { return fmt == GEMM_FMT_F32 ? 4 : 2; }

struct Range {
  uintptr_t lo, hi;
};

// Byte range of rows x row_bytes bytes with row stride ld; false on overflow.
bool byte_rows(const void* p, int64_t rows, int64_t ld, int64_t row_bytes, Range* r) {
  int64_t a;
  if (__builtin_mul_overflow(rows - 1, ld, &a) || __builtin_add_overflow(a, row_bytes, &a) ||
      a > INT64_MAX / 2)
    return false;
  r->lo = (uintptr_t)p;
  r->hi = r->lo + (uintptr_t)a;
  return r->hi >= r->lo;
}

bool overlap(const Range& a, const Range& b) { return ranges_overlap(a.lo, a.hi, b.lo, b.hi); }

int run(const void* fn, dim3 grid, int threads, void* args, hipStream_t s) {
  void* p[] = {args};
  return hipLaunchKernel(fn, grid, dim3((unsigned)threads), p, 0, s) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

// Data and scale arrays of an MX4 matrix of `rows` rows.
int check_mx4(const void* data, int64_t ldd, const void* scales, int64_t lds, int64_t rows, int64_t K,
              Range* rd, Range* rs) {
  const int64_t kb = cdiv(K, kMxBlock);
  if (ldd <= 0 || lds <= 0) return GEMM_ERR_STRIDE;
  if (rows > 1 && (ldd < kb * kMxBytes || lds < kb)) return GEMM_ERR_STRIDE;
  if (!byte_rows(data, rows, ldd, kb * kMxBytes, rd) || !byte_rows(scales, rows, lds, kb, rs))
    return GEMM_ERR_SHAPE;
  if (((uintptr_t)data & 15u) || (rows > 1 && ldd % 16 != 0)) return GEMM_ERR_LAYOUT;
  return GEMM_OK;
}

// K up to 2^36, as the 16-bit tiles: chunk counters stay far inside int64.
constexpr int64_t kMaxK = INT64_C(1) << 36;

template <int XF, int DT, int NS, int MT, int UC>
int launch_strip(const StripArgs& a, hipStream_t s) {
  const int64_t gx = cdiv(a.N, 16 * NS), gy = cdiv(a.M, 16 * MT);
  if (gx > kMaxGrid || gy > 65535) return GEMM_ERR_SHAPE;
  StripArgs copy = a;
  return run((const void*)mx4_strip_kernel<XF, DT, NS, MT, UC>, dim3((unsigned)gx, (unsigned)gy),
             64 * kStripWaves, &copy, s);
}

template <int XF, int DT>
int launch_strip_m(const StripArgs& a, hipStream_t s) {
  if (a.M <= 16) return launch_strip<XF, DT, 1, 1, 2>(a, s);
  if (a.M <= 32) return launch_strip<XF, DT, 1, 2, 2>(a, s);
  return launch_strip<XF, DT, 2, 4, 1>(a, s);
}

}  // namespace

extern "C" {

int gemm_mx4_quantize(const void* X, int32_t fmt, int64_t ldx_g, int64_t ldx_r, int64_t ldx_k,
                      int64_t G, int64_t R, int64_t K, void* data, void* scales, void* stream) {
  if (!X || !data || !scales) return GEMM_ERR_NULL;
  if (G <= 0 || R <= 0 || K <= 0 || K > kMaxK) return GEMM_ERR_SHAPE;
  if (fmt < GEMM_FMT_F16 || fmt > GEMM_FMT_F32) return GEMM_ERR_OPTS;
  if (ldx_g <= 0 || ldx_r <= 0 || ldx_k <= 0) return GEMM_ERR_STRIDE;
  int64_t rk, gg, span, rows;
  if (!view_span(R, K, ldx_r, ldx_k, &rk) || __builtin_mul_overflow(G - 1, ldx_g, &gg) ||
      __builtin_add_overflow(rk, gg, &span) || span > INT64_MAX / 8 || __builtin_mul_overflow(G, R, &rows))
    return GEMM_ERR_SHAPE;
  const int64_t Kb = cdiv(K, kMxBlock);
  Range rx{(uintptr_t)X, (uintptr_t)X + (uintptr_t)((span + 1) * elem_size(fmt))}, rd, rs;
  if (rx.hi < rx.lo) return GEMM_ERR_SHAPE;
  const int rc = check_mx4(data, Kb * kMxBytes, scales, Kb, rows, K, &rd, &rs);
  if (rc) return rc;
  if (overlap(rx, rd) || overlap(rx, rs) || overlap(rd, rs)) return GEMM_ERR_ALIAS;

  QuantArgs a{X, ldx_g, ldx_r, ldx_k, G, R, K, (uint8_t*)data, (uint8_t*)scales, Kb, 1, 1};
  int64_t waves;
  const void* fn;
  if (ldx_k == 1) {
    // Dense rows of whole blocks are one long row.
    if (K % kMxBlock == 0 && ldx_r == K && (G == 1 || ldx_g == R * K)) {
      a.G = a.R = 1;
      a.K = rows * K;
      a.Kb = rows * Kb;
    }
    const int64_t octs = 4 * a.Kb;
    a.segs = cdiv(octs, 64 * kQuantU);
    a.rpw = octs <= 32 ? (int32_t)(64 / octs) : 1;
    waves = a.rpw > 1 ? cdiv(a.G * a.R, a.rpw) : a.G * a.R * a.segs;
    fn = fmt == GEMM_FMT_F16    ? (const void*)quantize_rows_kernel<MX_F16>
         : fmt == GEMM_FMT_BF16 ? (const void*)quantize_rows_kernel<MX_BF16>
                                : (const void*)quantize_rows_kernel<MX_F32>;
  } else {
    waves = cdiv(rows, 64) * Kb;
    fn = fmt == GEMM_FMT_F16    ? (const void*)quantize_columns_kernel<MX_F16>
         : fmt == GEMM_FMT_BF16 ? (const void*)quantize_columns_kernel<MX_BF16>
                                : (const void*)quantize_columns_kernel<MX_F32>;
  }
  const int64_t grid = cdiv(waves, 4);
  if (grid > kMaxGrid) return GEMM_ERR_SHAPE;
  return run(fn, dim3((unsigned)grid), 256, &a, (hipStream_t)stream);
}

int gemm_mx4_dequantize(const void* data, int64_t ldd, const void* scales, int64_t lds, int64_t R,
                        int64_t K, void* Y, int32_t fmt, int64_t ldy, void* stream) {
  if (!data || !scales || !Y) return GEMM_ERR_NULL;
  if (R <= 0 || K <= 0 || K > kMaxK) return GEMM_ERR_SHAPE;
  if (fmt < GEMM_FMT_F16 || fmt > GEMM_FMT_F32) return GEMM_ERR_OPTS;
  if (ldy < K) return GEMM_ERR_LDC;
  Range rd, rs;
  const int rc = check_mx4(data, ldd, scales, lds, R, K, &rd, &rs);
  if (rc) return rc;
  int64_t span;
  if (!view_span(R, K, ldy, 1, &span) || span > INT64_MAX / 8) return GEMM_ERR_SHAPE;
  const Range ry{(uintptr_t)Y, (uintptr_t)Y + (uintptr_t)((span + 1) * elem_size(fmt))};
  if (ry.hi < ry.lo) return GEMM_ERR_SHAPE;
  if (overlap(ry, rd) || overlap(ry, rs)) return GEMM_ERR_ALIAS;

  DequantArgs a{(const uint8_t*)data, ldd, (const uint8_t*)scales, lds, R, K, Y, ldy, 1, 1};
  const int64_t kb = cdiv(K, kMxBlock);
  if (K % kMxBlock == 0 && ldy == K && ldd == kb * kMxBytes && lds == kb) {   // one long row
    a.R = 1;
    a.K = R * K;
  }
  const int64_t octs = cdiv(a.K, 8);
  a.segs = cdiv(octs, 64 * kQuantU);
  a.rpw = octs <= 32 ? (int32_t)(64 / octs) : 1;
  const int64_t waves = a.rpw > 1 ? cdiv(a.R, a.rpw) : a.R * a.segs;
  const int64_t grid = cdiv(waves, 4);
  if (grid > kMaxGrid) return GEMM_ERR_SHAPE;
  const void* fn = fmt == GEMM_FMT_F16    ? (const void*)dequantize_kernel<MX_F16>
                   : fmt == GEMM_FMT_BF16 ? (const void*)dequantize_kernel<MX_BF16>
                                          : (const void*)dequantize_kernel<MX_F32>;
  return run(fn, dim3((unsigned)grid), 256, &a, (hipStream_t)stream);
}

size_t gemm_mx4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  (void)M; (void)N; (void)K;
  return 0;
}

int gemm_mx4(const void* A, int64_t lda, const void* SA, int64_t ldsa, const void* B, int64_t ldb,
             const void* SB, int64_t ldsb, void* C, int32_t fmt_c, int64_t ldc, int64_t M, int64_t N,
             int64_t K, void* stream, void* workspace, size_t workspace_bytes) {
  (void)workspace; (void)workspace_bytes;
  if (!A || !SA || !B || !SB || !C) return GEMM_ERR_NULL;
  if (M <= 0 || N <= 0 || K <= 0 || K > kMaxK) return GEMM_ERR_SHAPE;
  if (fmt_c != GEMM_FMT_F16 && fmt_c != GEMM_FMT_BF16) return GEMM_ERR_OPTS;
  if (ldc < N) return GEMM_ERR_LDC;
  Range ra, rsa, rb, rsb, rc_;
  int rc = check_mx4(A, lda, SA, ldsa, M, K, &ra, &rsa);
  if (rc) return rc;
  if ((rc = check_mx4(B, ldb, SB, ldsb, N, K, &rb, &rsb))) return rc;
  int64_t span;
  if (!view_span(M, N, ldc, 1, &span) || !byte_rows(C, 1, 1, 2 * (span + 1), &rc_)) return GEMM_ERR_SHAPE;
  if (overlap(rc_, ra) || overlap(rc_, rsa) || overlap(rc_, rb) || overlap(rc_, rsb)) return GEMM_ERR_ALIAS;
  const StripArgs a{(const char*)A, lda, (const uint8_t*)SA, ldsa, (const char*)B, ldb, (const uint8_t*)SB,
                    ldsb, (uint16_t*)C, ldc, M, N, K};
  return fmt_c == GEMM_FMT_F16 ? launch_strip_m<SX_MX4, DT_F16>(a, (hipStream_t)stream)
                               : launch_strip_m<SX_MX4, DT_BF16>(a, (hipStream_t)stream);
}

int gemm_mx4_a16(const void* A, int32_t fmt, int64_t lda, const void* B, int64_t ldb, const void* SB,
                 int64_t ldsb, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K, void* stream) {
  if (!A || !B || !SB || !C) return GEMM_ERR_NULL;
  if (M <= 0 || N <= 0 || K <= 0 || K > kMaxK) return GEMM_ERR_SHAPE;
  if (fmt != GEMM_FMT_F16 && fmt != GEMM_FMT_BF16) return GEMM_ERR_OPTS;
  if (lda <= 0) return GEMM_ERR_STRIDE;
  if (ldc < N) return GEMM_ERR_LDC;
  Range ra, rb, rsb, rc_;
  int64_t span, spanA;
  if (!view_span(M, K, lda, 1, &spanA) || !byte_rows(A, 1, 1, 2 * (spanA + 1), &ra) ||
      !view_span(M, N, ldc, 1, &span) || !byte_rows(C, 1, 1, 2 * (span + 1), &rc_))
    return GEMM_ERR_SHAPE;
  const int rc = check_mx4(B, ldb, SB, ldsb, N, K, &rb, &rsb);
  if (rc) return rc;
  if (overlap(rc_, ra) || overlap(rc_, rb) || overlap(rc_, rsb)) return GEMM_ERR_ALIAS;
  const StripArgs a{(const char*)A, 2 * lda, nullptr, 0, (const char*)B, ldb, (const uint8_t*)SB, ldsb,
                    (uint16_t*)C, ldc, M, N, K};
  return fmt == GEMM_FMT_F16 ? launch_strip_m<SX_F16, DT_F16>(a, (hipStream_t)stream)
                             : launch_strip_m<SX_BF16, DT_BF16>(a, (hipStream_t)stream);
}

}  // extern "C"
