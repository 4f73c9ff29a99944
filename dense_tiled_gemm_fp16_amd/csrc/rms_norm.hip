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

// How a row lies in registers: octets per lane (U), waves, lanes of a wave.
struct Shape {
  int U, waves, lanes;   // lanes: log2
  int per() const { return waves > 1 ? 1 : 4 * (64 >> lanes); }   // rows of a workgroup
  int threads() const { return waves > 1 ? 64 * waves : 256; }
};

// Short rows: one octet a lane, in as few lanes as hold the row's blocks.  Others
// two, or more where `most` waves would not hold the row.
Shape shape(int64_t K, int most) {
  const int64_t octs = cdiv(K, 8);
  if (octs <= 64) return Shape{1, 1, octs <= 16 ? 4 : octs <= 32 ? 5 : 6};
  int U = 2;
  while (cdiv(octs, 64 * U) > most && U < 8) U *= 2;
  return Shape{U, (int)cdiv(octs, 64 * U), 6};
}
Shape norm_shape(int64_t K) { return shape(K, 16); }
// The backward kernel holds more of a row: 8 waves, and rows wider than they hold
// have a kernel of their own (U 8, 16 waves).
Shape back_shape(int64_t K) {
  const Shape s = shape(K, kBackThreads / 64);
  return s.U < kWideOcts ? s : Shape{kWideOcts, kWideThreads / 64, 6};
}

bool weight_format(int32_t fmt, int32_t fmt_w) { return fmt_w == fmt || fmt_w == GEMM_FMT_F32; }

// A kernel's last three template arguments (residual or dh, float32 weight, rows
// past the caches) from as many truth values.
#define GEMM_BY_FLAGS2(KERNEL, b, c, ...)                                                                          \
  ((b) ? ((c) ? (const void*)KERNEL<__VA_ARGS__, true, true> : (const void*)KERNEL<__VA_ARGS__, true, false>)         \
       : ((c) ? (const void*)KERNEL<__VA_ARGS__, false, true> : (const void*)KERNEL<__VA_ARGS__, false, false>))
#define GEMM_BY_FLAGS(KERNEL, a, b, c, ...)                                                                        \
  ((a) ? GEMM_BY_FLAGS2(KERNEL, b, c, __VA_ARGS__, true) : GEMM_BY_FLAGS2(KERNEL, b, c, __VA_ARGS__, false))

// Past the caches: 32768 x 7168 bfloat16 with a residual 276 us instead of 288, the
// gradients of 16384 x 7168 with dh 165 instead of 184 (one run, two sets in turn).
bool once(int64_t R, int64_t K, int bytes) { return (double)R * (double)K * bytes > kOnceBytes; }

template <int FMT, int F8>
const void* norm_fn2(int U, bool res, bool w32, bool o) {
  return U == 1   ? GEMM_BY_FLAGS(rms_norm_f8_kernel, res, w32, o, FMT, F8, 1)
         : U == 2 ? GEMM_BY_FLAGS(rms_norm_f8_kernel, res, w32, o, FMT, F8, 2)
         : U == 4 ? GEMM_BY_FLAGS(rms_norm_f8_kernel, res, w32, o, FMT, F8, 4)
                  : GEMM_BY_FLAGS(rms_norm_f8_kernel, res, w32, o, FMT, F8, 8);
}
const void* norm_fn(int32_t fmt, int32_t fmt8, int U, bool res, bool w32, bool o) {
  if (fmt == GEMM_FMT_F16)
    return fmt8 == 0 ? norm_fn2<MX_F16, F8_E4M3>(U, res, w32, o) : norm_fn2<MX_F16, F8_E5M2>(U, res, w32, o);
  return fmt8 == 0 ? norm_fn2<MX_BF16, F8_E4M3>(U, res, w32, o) : norm_fn2<MX_BF16, F8_E5M2>(U, res, w32, o);
}

template <int FMT, bool TAIL>
const void* back_fn2(int U, bool dh, bool w32, bool o) {
  return U == 1   ? GEMM_BY_FLAGS(rms_norm_back_kernel, dh, w32, o, FMT, 1, TAIL)
         : U == 2 ? GEMM_BY_FLAGS(rms_norm_back_kernel, dh, w32, o, FMT, 2, TAIL)
                  : GEMM_BY_FLAGS(rms_norm_back_kernel, dh, w32, o, FMT, 4, TAIL);
}
template <int FMT>
const void* back_fn1(int U, bool tail, bool dh, bool w32, bool o) {
  if (U > 4) return GEMM_BY_FLAGS2(rms_norm_back_wide_kernel, dh, w32, FMT);
  return tail ? back_fn2<FMT, true>(U, dh, w32, o) : back_fn2<FMT, false>(U, dh, w32, o);
}
const void* back_fn(int32_t fmt, int U, bool tail, bool dh, bool w32, bool o) {
  return fmt == GEMM_FMT_F16 ? back_fn1<MX_F16>(U, tail, dh, w32, o) : back_fn1<MX_BF16>(U, tail, dh, w32, o);
}

template <int COLS>
const void* dw_fn1(int32_t fmt_w) {
  return fmt_w == GEMM_FMT_F32   ? (const void*)rms_norm_dw_kernel<MX_F32, COLS>
         : fmt_w == GEMM_FMT_F16 ? (const void*)rms_norm_dw_kernel<MX_F16, COLS>
                                 : (const void*)rms_norm_dw_kernel<MX_BF16, COLS>;
}
const void* dw_fn(int32_t fmt_w, int cols) { return cols == 16 ? dw_fn1<16>(fmt_w) : dw_fn1<64>(fmt_w); }

// Workgroups of the backward kernel: each leaves a row of sums per row that it
// takes at a time, so no more than are needed to fill 256 compute units, and at
// least two rows for each (16384 x 512 bfloat16: 28.9 us with 512 workgroups of 4
// rows).  Rows of several waves: as many workgroups a unit as have 12288 elements
// between them, two at least, and as many at most as find room by their registers
// (norm_kernel.hpp): of up to two octets four waves a SIMD, though of 5 waves and more
// two workgroups; of four octets two waves a SIMD, and of the wide kernel's 1024 lanes,
// one workgroup.  9698 x 3480: 57 us with two a unit, 46 with four; 12000 x 5000: 83
// with two, 103 with three; twice as many as find room, a second round of them half
// empty: 4000 x 12288 with dh 86 instead of 83, 2048 x 20000 113 instead of 97, 1000 x
// 65536 233 instead of 183, and twice the rows of sums.
int64_t back_grid(int64_t R, int64_t K, const Shape& s) {
  const int64_t room = s.U > 2 ? 1 : s.waves <= 4 ? 16 / s.waves : 2;
  const int64_t fill = s.waves == 1 ? std::max<int64_t>(512, (INT64_C(2) << 20) / K)
                                    : 256 * std::min<int64_t>(room, std::max<int64_t>(2, cdiv(12288, K)));
  const int64_t parts = std::min<int64_t>(fill, std::max<int64_t>(cdiv(R, 4), std::min<int64_t>(cdiv(R, 2), 512)));
  return std::max<int64_t>(parts / s.per(), 1);
}

// `out` may be `in` itself, element for element; other overlaps are refused.
bool clash(const Range& out, const Range& in, const void* po, int64_t ldo, const void* pi, int64_t ldi, int64_t R) {
  return overlap(out, in) && !(po == pi && (ldo == ldi || R == 1));
}

}  // namespace

extern "C" {

int gemm_rms_norm_f8(const gemm_rms_norm_f8_args* args, void* stream) {
  if (!args) return GEMM_ERR_NULL;
  const auto [X, ldx, residual, ldr, W, H, ldh, data, ldd, scales, lds_r, lds_k, R, K, eps, fmt, fmt_w, fmt8] = *args;
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
  if (!apart(R, cdiv(K, kF8Block), lds_r, lds_k)) return GEMM_ERR_LDC;
  if ((uintptr_t)scales & 3u) return GEMM_ERR_LAYOUT;
  if (overlap(rd, rx) || overlap(rd, rw) || overlap(rd, rs) || overlap(rs, rx) || overlap(rs, rw)) return GEMM_ERR_ALIAS;
  if (residual && (overlap(rd, rr) || overlap(rs, rr) || overlap(rd, rh) || overlap(rs, rh) || overlap(rh, rw) ||
                   clash(rh, rx, H, ldh, X, ldx, R) || clash(rh, rr, H, ldh, residual, ldr, R)))
    return GEMM_ERR_ALIAS;
  const Shape sh = norm_shape(K);
  const int64_t grid = cdiv(R, sh.per());
  if (!fits_x(grid, sh.threads())) return GEMM_ERR_SHAPE;
  NormArgs a{X, ldx, residual, ldr, W, H, ldh, (uint8_t*)data, ldd, scales, lds_r, lds_k, R, K, eps, sh.waves, sh.lanes};
  return run(norm_fn(fmt, fmt8, sh.U, residual != nullptr, fmt_w == GEMM_FMT_F32,
                     once(R, K, residual ? 7 : 3)),
             dim3((unsigned)grid),
             sh.threads(), &a, (hipStream_t)stream);
}

size_t gemm_rms_norm_backward_workspace_bytes(int64_t R, int64_t K) {
  if (R <= 0 || K <= 0 || K > kMaxNormK) return 0;
  const Shape sh = back_shape(K);
  return (size_t)(back_grid(R, K, sh) * sh.per() * K * 4);
}

int gemm_rms_norm_backward(const gemm_rms_norm_backward_args* args, void* stream, void* workspace,
                           size_t workspace_bytes) {
  if (!args) return GEMM_ERR_NULL;
  const auto [DY, ldy, H, ldh, W, DH, lddh, DX, lddx, DW, R, K, eps, fmt, fmt_w] = *args;
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
  const Shape sh = back_shape(K);
  const int64_t grid = back_grid(R, K, sh);
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
  NormBackArgs a{DY, ldy, H, ldh, W, DH, lddh, DX, lddx, (float*)ws.get(), R, K, eps, sh.waves, sh.lanes};
  rc = run(back_fn(fmt, sh.U, K % 8 != 0, DH != nullptr, fmt_w == GEMM_FMT_F32, once(R, K, DH ? 8 : 6)), dim3((unsigned)grid), sh.threads(), &a, s);
  if (rc == GEMM_OK) {
    const float* part = a.part;
    int64_t parts = grid * sh.per(), k = K;
    void* dw = DW;
    void* p[] = {&part, &parts, &k, &dw};
    const int cols = K < 4096 ? 16 : 64;
    const void* fn = dw_fn(fmt_w, cols);
    if (hipLaunchKernel(fn, dim3((unsigned)cdiv(K, cols)), dim3(1024), p, 0, s) != hipSuccess) rc = GEMM_ERR_HIP;
  }
  return ws.done(rc);
}

}  // extern "C"
