// Host side of include/rms_norm_f8.h: argument validation and launches of the
// norm and of its gradients.  Everything is checked before the first HIP call,
// so on any error nothing is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/rms_norm_f8.h"
#include "host_launch.hpp"
#include "norm_kernel.hpp"

using namespace gemmf16;

namespace {

constexpr int64_t kMaxNormK = 65536;   // 16 waves of 8 octets a lane

// Octets per lane (U) and waves of a row: two octets while 16 waves hold the
// row.
void norm_shape(int64_t K, int* U, int* waves) {
  const int64_t octs = cdiv(K, 8);
  *U = 2;
  while (cdiv(octs, 64 * *U) > 16) *U *= 2;
  *waves = (int)cdiv(octs, 64 * *U);
}

bool weight_format(int32_t fmt, int32_t fmt_w) { return fmt_w == fmt || fmt_w == GEMM_FMT_F32; }

template <int FMT, int F8, int U>
const void* norm_fn3(bool res, bool w32) {
  if (res) return w32 ? (const void*)rms_norm_f8_kernel<FMT, F8, U, true, true> : (const void*)rms_norm_f8_kernel<FMT, F8, U, true, false>;
  return w32 ? (const void*)rms_norm_f8_kernel<FMT, F8, U, false, true> : (const void*)rms_norm_f8_kernel<FMT, F8, U, false, false>;
}
template <int FMT, int F8>
const void* norm_fn2(int U, bool res, bool w32) {
  return U == 2 ? norm_fn3<FMT, F8, 2>(res, w32) : U == 4 ? norm_fn3<FMT, F8, 4>(res, w32) : norm_fn3<FMT, F8, 8>(res, w32);
}
const void* norm_fn(int32_t fmt, int32_t fmt8, int U, bool res, bool w32) {
  if (fmt == GEMM_FMT_F16)
    return fmt8 == 0 ? norm_fn2<MX_F16, F8_E4M3>(U, res, w32) : norm_fn2<MX_F16, F8_E5M2>(U, res, w32);
  return fmt8 == 0 ? norm_fn2<MX_BF16, F8_E4M3>(U, res, w32) : norm_fn2<MX_BF16, F8_E5M2>(U, res, w32);
}

template <int FMT, int U>
const void* back_fn2(bool dh, bool w32) {
  if (dh) return w32 ? (const void*)rms_norm_back_kernel<FMT, U, true, true> : (const void*)rms_norm_back_kernel<FMT, U, true, false>;
  return w32 ? (const void*)rms_norm_back_kernel<FMT, U, false, true> : (const void*)rms_norm_back_kernel<FMT, U, false, false>;
}
const void* back_fn(int32_t fmt, int U, bool dh, bool w32) {
  if (fmt == GEMM_FMT_F16)
    return U == 2 ? back_fn2<MX_F16, 2>(dh, w32) : U == 4 ? back_fn2<MX_F16, 4>(dh, w32) : back_fn2<MX_F16, 8>(dh, w32);
  return U == 2 ? back_fn2<MX_BF16, 2>(dh, w32) : U == 4 ? back_fn2<MX_BF16, 4>(dh, w32) : back_fn2<MX_BF16, 8>(dh, w32);
}

// Workgroups of the backward kernel and the rows that each takes at a time.
void back_grid(int64_t R, int waves, int64_t* grid, int64_t* per) {
  *per = waves == 1 ? 4 : 1;
  *grid = std::min<int64_t>(cdiv(R, *per), 512);
}

// `out` may be `in` itself, element for element; other overlaps are refused.
bool clash(const Range& out, const Range& in, const void* po, int64_t ldo, const void* pi, int64_t ldi, int64_t R) {
  return overlap(out, in) && !(po == pi && (ldo == ldi || R == 1));
}

}  // namespace

extern "C" {

int gemm_rms_norm_f8(const void* X, int64_t ldx, const void* residual, int64_t ldr, int32_t fmt, const void* W,
                     int32_t fmt_w, float eps, void* H, int64_t ldh, void* data, int32_t fmt8, int64_t ldd,
                     float* scales, int64_t lds_r, int64_t lds_k, int64_t R, int64_t K, void* stream) {
  if (!X || !W || !data || !scales || (residual && !H)) return GEMM_ERR_NULL;
  if (R <= 0 || K <= 0 || K > kMaxNormK) return GEMM_ERR_SHAPE;
  if ((fmt != GEMM_FMT_F16 && fmt != GEMM_FMT_BF16) || !weight_format(fmt, fmt_w) || fmt8 < 0 || fmt8 > 1 || !(eps >= 0.0f))
    return GEMM_ERR_OPTS;
  if (ldx <= 0 || (residual && ldr <= 0) || lds_r <= 0 || lds_k <= 0) return GEMM_ERR_STRIDE;
  if (ldd < K || (residual && ldh < K)) return GEMM_ERR_LDC;
  Range rx, rr{}, rw, rh{}, rd, rs;
  if (!byte_view(X, R, K, ldx, 1, 2, &rx) || !byte_rows(W, 1, 1, K * (fmt_w == GEMM_FMT_F32 ? 4 : 2), &rw) ||
      !byte_rows(data, R, ldd, K, &rd) || !byte_view(scales, R, cdiv(K, kF8Block), lds_r, lds_k, 4, &rs))
    return GEMM_ERR_SHAPE;
  if (residual && (!byte_view(residual, R, K, ldr, 1, 2, &rr) || !byte_view(H, R, K, ldh, 1, 2, &rh))) return GEMM_ERR_SHAPE;
  if ((uintptr_t)scales & 3u) return GEMM_ERR_LAYOUT;
  if (overlap(rd, rx) || overlap(rd, rw) || overlap(rd, rs) || overlap(rs, rx) || overlap(rs, rw)) return GEMM_ERR_ALIAS;
  if (residual && (overlap(rd, rr) || overlap(rs, rr) || overlap(rd, rh) || overlap(rs, rh) || overlap(rh, rw) ||
                   clash(rh, rx, H, ldh, X, ldx, R) || clash(rh, rr, H, ldh, residual, ldr, R)))
    return GEMM_ERR_ALIAS;
  int U, waves;
  norm_shape(K, &U, &waves);
  const int per = waves == 1 ? 4 : 1;
  const int64_t grid = cdiv(R, per);
  if (!fits_x(grid, 64 * waves * per)) return GEMM_ERR_SHAPE;
  NormArgs a{X, ldx, residual, ldr, W, H, ldh, (uint8_t*)data, ldd, scales, lds_r, lds_k, R, K, eps, waves};
  return run(norm_fn(fmt, fmt8, U, residual != nullptr, fmt_w == GEMM_FMT_F32), dim3((unsigned)grid),
             64 * waves * per, &a, (hipStream_t)stream);
}

size_t gemm_rms_norm_backward_workspace_bytes(int64_t R, int64_t K) {
  if (R <= 0 || K <= 0 || K > kMaxNormK) return 0;
  int U, waves;
  int64_t grid, per;
  norm_shape(K, &U, &waves);
  back_grid(R, waves, &grid, &per);
  return (size_t)(grid * per * K * 4);
}

int gemm_rms_norm_backward(const void* DY, int64_t ldy, const void* H, int64_t ldh, int32_t fmt, const void* W,
                           int32_t fmt_w, float eps, const void* DH, int64_t lddh, void* DX, int64_t lddx, void* DW,
                           int64_t R, int64_t K, void* stream, void* workspace, size_t workspace_bytes) {
  if (!DY || !H || !W || !DX || !DW) return GEMM_ERR_NULL;
  if (R <= 0 || K <= 0 || K > kMaxNormK) return GEMM_ERR_SHAPE;
  if ((fmt != GEMM_FMT_F16 && fmt != GEMM_FMT_BF16) || !weight_format(fmt, fmt_w) || !(eps >= 0.0f)) return GEMM_ERR_OPTS;
  if (ldy <= 0 || ldh <= 0 || (DH && lddh <= 0)) return GEMM_ERR_STRIDE;
  if (lddx < K) return GEMM_ERR_LDC;
  const int64_t wb = K * (fmt_w == GEMM_FMT_F32 ? 4 : 2);
  Range ry, rh, rw, rd{}, rx, rdw;
  if (!byte_view(DY, R, K, ldy, 1, 2, &ry) || !byte_view(H, R, K, ldh, 1, 2, &rh) || !byte_rows(W, 1, 1, wb, &rw) ||
      !byte_view(DX, R, K, lddx, 1, 2, &rx) || !byte_rows(DW, 1, 1, wb, &rdw) ||
      (DH && !byte_view(DH, R, K, lddh, 1, 2, &rd)))
    return GEMM_ERR_SHAPE;
  if (clash(rx, ry, DX, lddx, DY, ldy, R) || overlap(rx, rh) || overlap(rx, rw) || overlap(rx, rdw) ||
      (DH && clash(rx, rd, DX, lddx, DH, lddh, R)) || overlap(rdw, ry) || overlap(rdw, rh) || overlap(rdw, rw) ||
      (DH && overlap(rdw, rd)))
    return GEMM_ERR_ALIAS;
  int U, waves;
  int64_t grid, per;
  norm_shape(K, &U, &waves);
  back_grid(R, waves, &grid, &per);
  const size_t need = gemm_rms_norm_backward_workspace_bytes(R, K);
  if (workspace) {
    const Range rws{(uintptr_t)workspace, (uintptr_t)workspace + need};
    if (overlap(rws, ry) || overlap(rws, rh) || overlap(rws, rw) || overlap(rws, rx) || overlap(rws, rdw) ||
        (DH && overlap(rws, rd)))
      return GEMM_ERR_ALIAS;
  }
  hipStream_t s = (hipStream_t)stream;
  Workspace ws;
  int rc = ws.take(workspace, workspace_bytes, need, s);
  if (rc) return rc;
  NormBackArgs a{DY, ldy, H, ldh, W, DH, lddh, DX, lddx, (float*)ws.get(), R, K, eps, waves};
  rc = run(back_fn(fmt, U, DH != nullptr, fmt_w == GEMM_FMT_F32), dim3((unsigned)grid), (int)(64 * waves * per), &a, s);
  if (rc == GEMM_OK) {
    const float* part = a.part;
    int64_t parts = grid * per, k = K;
    void* p[] = {&part, &parts, &k, &DW};
    const void* fn = fmt_w == GEMM_FMT_F32   ? (const void*)rms_norm_dw_kernel<MX_F32>
                     : fmt_w == GEMM_FMT_F16 ? (const void*)rms_norm_dw_kernel<MX_F16>
                                             : (const void*)rms_norm_dw_kernel<MX_BF16>;
    if (hipLaunchKernel(fn, dim3((unsigned)cdiv(K, 64)), dim3(1024), p, 0, s) != hipSuccess) rc = GEMM_ERR_HIP;
  }
  return ws.done(rc);
}

}  // extern "C"
