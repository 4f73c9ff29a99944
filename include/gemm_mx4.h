/*
 * gemm_mx4.h -- microscaled 4-bit floating point (OCP MX FP4) on MI355X:
 * quantisation, and products with 4-bit weights.  Same library, return codes
 * (enum gemm_status), stream and workspace rules as gemm_f16.h.
 *
 * An MX4 matrix [R, K] is two byte arrays:
 *     data    R rows of 16 * ceil(K/32) bytes: element k in the low (k even)
 *             or high (k odd) half of byte k/2; 1 sign, 2 exponent and 1
 *             mantissa bits: +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}
 *     scales  R rows of ceil(K/32) bytes: block b (elements 32b .. 32b+31)
 *             is multiplied by 2^(scale - 127); 255 makes the block NaN
 * Row strides ldd and lds are in bytes, at least the row's bytes.  The
 * elements of the last block past K count as absent: the quantiser writes
 * zeros there and the products multiply them by zero (their scale is the
 * block's, so a NaN block is NaN).
 *
 * Results are deterministic: sums run in a fixed order, without atomics.
 */
#ifndef GEMM_MX4_H
#define GEMM_MX4_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element formats of 16- and 32-bit operands below. */
enum gemm_mx4_format { GEMM_FMT_F16 = 0, GEMM_FMT_BF16 = 1, GEMM_FMT_F32 = 2 };

/*
 * Quantise G stacked matrices X[g,r,k] at X + g*ldx_g + r*ldx_r + k*ldx_k
 * (elements of format fmt, strides in elements, positive) along k.  Row
 * g*R + r of the output is at data + (g*R + r) * 16*ceil(K/32) and
 * scales + (g*R + r) * ceil(K/32): no padding between rows.
 *
 * With m the block's largest magnitude the scale is 2^(floor(log2 m) - 2),
 * at least 2^-127 (which a zero block gets); elements are divided by it and
 * rounded to nearest, ties to the even code, saturating at 6.  A block that
 * holds an infinity or a NaN gets scale 255 (and zero codes).
 * data is 16-byte aligned.
 */
int gemm_mx4_quantize(const void* X, int32_t fmt, int64_t ldx_g, int64_t ldx_r, int64_t ldx_k,
                      int64_t G, int64_t R, int64_t K, void* data, void* scales, void* stream);

/* Y[r,k] at Y + r*ldy + k (elements of format fmt, ldy >= K) := the values
 * of an MX4 matrix, rounded once to nearest even. */
int gemm_mx4_dequantize(const void* data, int64_t ldd, const void* scales, int64_t lds, int64_t R,
                        int64_t K, void* Y, int32_t fmt, int64_t ldy, void* stream);

/*
 * C[m,n] := sum_k A[m,k] B[n,k] for MX4 A [M, K] and MX4 B [N, K], fp32
 * accumulation, C of format fmt_c (GEMM_FMT_F16 or GEMM_FMT_BF16), row-major
 * with row stride ldc.  lda, ldb, ldsa, ldsb: row strides of the data and
 * scale arrays in bytes; data rows are 16-byte aligned and, as the scales'
 * rows, at most 2^26 bytes apart (GEMM_ERR_LAYOUT).
 * Needs gemm_mx4_workspace_bytes(M, N, K) bytes of workspace (may be 0); with
 * workspace == NULL they are allocated in stream order.  GEMM_ERR_SHAPE: more
 * than 65535 * 64 rows of A against 128 rows of B or fewer, more than 2^27
 * rows of B against 128 rows of A or fewer, or 2^23 tiles of 256 x 256 and more.
 */
int gemm_mx4(const void* A, int64_t lda, const void* SA, int64_t ldsa, const void* B, int64_t ldb,
             const void* SB, int64_t ldsb, void* C, int32_t fmt_c, int64_t ldc, int64_t M, int64_t N,
             int64_t K, void* stream, void* workspace, size_t workspace_bytes);
size_t gemm_mx4_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * C[m,n] := sum_k A[m,k] B[n,k] for a 16-bit A (format fmt, GEMM_FMT_F16 or
 * GEMM_FMT_BF16; A[m,k] at A + m*lda + k) and MX4 B [N, K]; C has A's format.
 * The weights enter the products exactly, at any scale, with two exceptions:
 * beside a binary16 A those of scale 0, below 2^-124, count as zeros, and
 * values of 2^128 and more (codes of 4 and 6 at scale 253, of 2 and more at
 * scale 254, neither of which the quantiser gives) are past the range: the
 * outputs of their row are infinite or NaN.  (gemm_mx4 takes those exactly too.)
 * A kernel for few
 * rows (the weights are read once per 32 rows of A): with many rows, quantise
 * A and call gemm_mx4.  Rows of A at most 2^25 elements apart, rows of B as
 * above (GEMM_ERR_LAYOUT); M up to 65535 * 32, N up to 2^27 (GEMM_ERR_SHAPE).
 */
int gemm_mx4_a16(const void* A, int32_t fmt, int64_t lda, const void* B, int64_t ldb, const void* SB,
                 int64_t ldsb, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_MX4_H */
