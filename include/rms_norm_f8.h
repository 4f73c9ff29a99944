/*
 * rms_norm_f8.h -- root-mean-square norm with the residual's addition and its
 * result in 8 bits (the input of gemm_f8s), and the norm's gradients, on MI355X.
 * Same library, return codes (enum gemm_status), stream and workspace rules as
 * gemm_f16.h; formats of enum gemm_mx4_format.
 *
 * Rows have unit stride along K and row strides in elements; K at most 65536.
 * Results are deterministic: sums run in a fixed order, without atomics.
 */
#ifndef RMS_NORM_F8_H
#define RMS_NORM_F8_H

#include "gemm_f8_scaled.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * h := x + residual, each row of K elements of format fmt (GEMM_FMT_F16 or
 * GEMM_FMT_BF16), rounded to it; or h = x with residual == NULL (then the H
 * argument is not used).
 * y := h * w / sqrt(mean(h^2) + eps) in float32, quantised by row blocks of 128 into
 * data and scales as gemm_f8s_quantize does a float32 X.  y is not stored; all is
 * float32, so a row of h whose squares sum past 3.4e38 becomes zeros, and with eps 0
 * one whose squares are all 0 has NaN scales.
 * w: K elements of fmt_w, GEMM_FMT_F32 or fmt.  H may be X or the residual
 * itself, at the same row stride; nothing else overlaps.
 */
typedef struct gemm_rms_norm_f8_args {
  const void* X;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* W;
  void* H;
  int64_t ldh;
  void* data;
  int64_t ldd;
  float* scales;
  int64_t lds_r, lds_k;
  int64_t R, K;
  float eps;
  int32_t fmt, fmt_w, fmt8;
} gemm_rms_norm_f8_args;

int gemm_rms_norm_f8(const gemm_rms_norm_f8_args* args, void* stream);

/*
 * Gradients of h and w, given those of y (DY) and, from the residual stream, of
 * h itself (DH, or NULL): with r = 1 / sqrt(mean(h^2) + eps) and g = DY * w,
 *     DX[row] := r (g - h r^2 mean(g h)) + DH[row]       (of x and the residual)
 *     DW[k]   := sum over rows of DY[row,k] h[row,k] r   (of fmt_w)
 * All is float32: a row of h whose squares sum past 3.4e38 has r = 0, and a DX of DH or
 * NaN.  DX may be DY or DH itself, at the same row stride.
 * Needs gemm_rms_norm_backward_workspace_bytes(R, K) bytes of workspace, 256-byte
 * aligned; with workspace == NULL they are allocated in stream order.
 */
typedef struct gemm_rms_norm_backward_args {
  const void* DY;
  int64_t ldy;
  const void* H;
  int64_t ldh;
  const void* W;
  const void* DH;
  int64_t lddh;
  void* DX;
  int64_t lddx;
  void* DW;
  int64_t R, K;
  float eps;
  int32_t fmt, fmt_w;
} gemm_rms_norm_backward_args;

int gemm_rms_norm_backward(const gemm_rms_norm_backward_args* args, void* stream, void* workspace,
                           size_t workspace_bytes);
size_t gemm_rms_norm_backward_workspace_bytes(int64_t R, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* RMS_NORM_F8_H */
