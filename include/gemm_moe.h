/*
 * gemm_moe.h -- a mixture-of-experts layer for a few tokens on MI355X: the
 * routing, the experts' gate and up products, the activation, the down
 * product and the weighted sum, in two kernels (three where few columns make
 * the weighted sum be split).  Same library, return codes
 * (enum gemm_status), stream and workspace rules as gemm_f16.h.
 *
 * For token t with row x_t of X [T, H] and logits L[t, 0 .. E-1]:
 *     S_t  = the top_k experts of the largest logits; equal logits go to the
 *            lower index, -inf never belongs, a NaN counts as the largest
 *     p_te = exp(L[t,e]) / sum_j exp(L[t,j]), j over S_t (renormalize != 0)
 *            or over all experts
 *     (g, u) = the first and the last I of W1[e] x_t,  W1[e] [2I, H]
 *     y_t  = sum over e in S_t of p_te W2[e] (silu(g) * u),  W2[e] [H, I]
 * with silu(g) = g / (1 + exp(-g)).  MX4 weights enter as in gemm_mx4_a16.  A token whose logits are all -inf gets
 * zeros.  Sums are fp32; silu(g) * u is carried as two bfloat16 parts (off by
 * at most 2^-16 of its value, at any magnitude), and Y is rounded once.  Results are deterministic: experts are added in ascending
 * order, without atomics on floating-point values; the order of a token's sums
 * depends on which experts the other tokens take.
 */
#ifndef GEMM_MOE_H
#define GEMM_MOE_H

#include "gemm_mx4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_MOE_MAX_TOKENS 64
#define GEMM_MOE_MAX_EXPERTS 512
#define GEMM_MOE_MAX_TOP_K 16

typedef struct {
  const void* X;        /* [T, H], format fmt (GEMM_FMT_F16 or GEMM_FMT_BF16)     */
  int64_t ldx;          /* row stride in elements                                */
  const void* logits;   /* [T, E], format fmt_logits (F16, BF16 or F32)           */
  int64_t ldl;          /* row stride in elements                                */
  const void* W1;       /* [E][2I, H]: 16-bit, of X's format, or MX4 data        */
  int64_t w1_e, w1_n;   /* expert and row strides: elements, or bytes with MX4   */
  const void* S1;       /* MX4 scales of W1 (NULL for 16-bit weights)            */
  int64_t s1_e, s1_n;   /* their strides in bytes                                */
  const void* W2;       /* [E][H, I], as W1                                      */
  int64_t w2_e, w2_n;
  const void* S2;
  int64_t s2_e, s2_n;
  void* Y;              /* [T, H], X's format                                    */
  int64_t ldy;          /* row stride in elements                                */
  int64_t T, E, H, I;   /* 1 <= T <= 64, 1 <= E <= 512                           */
  int32_t top_k;        /* 1 <= top_k <= min(E, 16)                              */
  int32_t fmt, fmt_logits;
  int32_t mx4;          /* 0: 16-bit weights, 1: MX4 weights                     */
  int32_t renormalize;
} gemm_moe_args;

/*
 * One layer.  Needs gemm_moe_workspace_bytes(T, E, top_k, H, I) bytes of
 * workspace, 256-byte aligned; with workspace == NULL they are allocated in
 * stream order.  GEMM_ERR_SHAPE: a size outside the bounds above (H up to
 * 2^26, I up to 2^20); GEMM_ERR_LAYOUT: the 2I rows of an expert's W1 or the T
 * rows of X span 4 GiB or more, or rows of W2 are 2^27 bytes or more apart.
 */
int gemm_moe(const gemm_moe_args* args, void* stream, void* workspace, size_t workspace_bytes);

/* Workspace bytes (0 for sizes outside the bounds). */
size_t gemm_moe_workspace_bytes(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_MOE_H */
