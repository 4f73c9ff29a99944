// Host side of include/gemm_f8_scaled.h: argument validation and launches of
// the quantiser and of the products scaled by blocks.  Everything is checked
// before the first HIP call, so on any error nothing is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_f8_scaled.h"
#include "f8s_convert.hpp"
#include "f8s_tiles.hpp"
#include "host_launch.hpp"

using namespace gemmf16;

namespace {

int64_t elem_size(int32_t fmt) { return fmt == GEMM_FMT_F32 ? 4 : 2; }

// K up to 2^36, as the other products.
constexpr int64_t kMaxK = INT64_C(1) << 36;

// How rows of octs octets are dealt to wave items; returns their number.
int64_t wave_items(int64_t rows, int64_t octs, int64_t* segs, Short* few) {
  *segs = cdiv(octs, kSlots);
  *few = Short{};
  if (*segs > 1 || rows == 1) return rows * *segs;
  *few = Short{(int32_t)octs, (int32_t)(kSlots / octs), (int32_t)(65536 / octs + 1)};
  return cdiv(rows, few->rows);
}

template <int FMT, int F8, bool ONCE>
const void* rows_fn(bool few) {
  return few ? (const void*)f8_rows_kernel<FMT, F8, true, ONCE> : (const void*)f8_rows_kernel<FMT, F8, false, ONCE>;
}
template <int FMT, int F8, bool ONCE>
const void* tiles_fn(bool square, bool along_k) {
  return !square ? (const void*)f8_tiles_kernel<FMT, F8, false, false, ONCE>
         : along_k ? (const void*)f8_tiles_kernel<FMT, F8, true, true, ONCE>
                   : (const void*)f8_tiles_kernel<FMT, F8, true, false, ONCE>;
}
template <int F8, bool ONCE>
const void* quant_fn(int32_t fmt, bool tiles, bool square, bool along_k, bool few) {
  if (tiles)
    return fmt == GEMM_FMT_F16    ? tiles_fn<MX_F16, F8, ONCE>(square, along_k)
           : fmt == GEMM_FMT_BF16 ? tiles_fn<MX_BF16, F8, ONCE>(square, along_k)
                                  : tiles_fn<MX_F32, F8, ONCE>(square, along_k);
  return fmt == GEMM_FMT_F16    ? rows_fn<MX_F16, F8, ONCE>(few)
         : fmt == GEMM_FMT_BF16 ? rows_fn<MX_BF16, F8, ONCE>(few)
                                : rows_fn<MX_F32, F8, ONCE>(few);
}
template <int F8>
const void* quant_fn(int32_t fmt, bool tiles, bool square, bool along_k, bool few, bool once) {
  return once ? quant_fn<F8, true>(fmt, tiles, square, along_k, few) : quant_fn<F8, false>(fmt, tiles, square, along_k, few);
}

const void* product_fn(int32_t fmt_a, int32_t fmt_b, int variant, bool rowb, bool wide, int out) {
  if (fmt_a == 0)
    return fmt_b == 0 ? f8s_fn<F8_E4M3, F8_E4M3>(variant, rowb, wide, out)
                      : f8s_fn<F8_E4M3, F8_E5M2>(variant, rowb, wide, out);
  return fmt_b == 0 ? f8s_fn<F8_E5M2, F8_E4M3>(variant, rowb, wide, out)
                    : f8s_fn<F8_E5M2, F8_E5M2>(variant, rowb, wide, out);
}

// Lanes reach a workgroup's rows by 32-bit offsets of bytes, scales too.
constexpr int64_t kMaxPitch = INT64_C(1) << 23, kMaxScalePitch = INT64_C(1) << 21;

// Whether a variant takes the call.
bool takes(const F8sArgs& a, int variant, bool wide) {
  if (variant == GEMM_F8S_TILE_256X256 && (a.shift == 0 || wide)) return false;
  const F8sShape& s = kF8sShapes[variant];
  const int64_t gm = cdiv(a.M, s.rows), gn = cdiv(a.N, s.cols);
  if (s.parts > 1) return gm <= 65535 && fits_x(gn, s.threads);
  int64_t grid;
  return !__builtin_mul_overflow(gm, gn, &grid) && fits_x(grid, s.threads);
}

// The variant that takes least by the times of f8s_tiles.hpp; 0 if none takes the
// call.  Measured in graphs (us; M x N x K, square blocks, bfloat16; strips of
// rows x columns, whose 8 waves share K, then tiles):
//   1 x 2048 x 7168      16x16 5.6, 16x32 5.7
//   32 x 7168 x 2048     16x32 6.4, 32x16 6.6, 32x32 4.6, 64x32 5.2
//   64 x 7168 x 2048     32x32 8.1, 64x32 5.5, 64x64 6.9, tile 64x128 12.9
//   128 x 2048 x 7168    32x32 8.8, 64x32 10.3, 64x64 12.7, tile 64x128 31
//   512 x 2048 x 7168    64x32 23, 64x64 17, tiles 64x128 30, 128x128 44
//   1024 x 2048 x 2048   64x64 12.0, tiles 64x128 11.3, 128x128 14.9
//   2048 x 2048 x 7168   64x64 59, tiles 64x128 45, 128x128 45, 256x256 76
//   2048 x 4096 x 4096   64x64 71, tiles 64x128 52, 128x128 41, 256x256 46
//   16384 x 4096 x 128   64x64 197, tiles 64x128 51, 128x128 35, 256x256 36
//   20864 x 1664 x 224   64x64 126, tiles 64x128 36, 128x128 28, 256x256 40
//   8192 x 2048 x 7168   64x64 226, tiles 64x128 169, 128x128 131, 256x256 100
//   32768 x 2048 x 7168  256x256 415
// Row blocks and float32: 2048 x 7168 x 8192 strips 64x64 312, tiles 64x128 297,
// 128x128 249; 512 x 2048 x 7168 22, 45, 67.  Over 74 sizes, most of them random,
// the choice took 2% longer than the best one in the mean, 16% at most.
int plan(const F8sArgs& a, bool wide, int cus) {
  int best = 0;
  float least = 0.0f;
  for (int v = 1; v < kF8sVariants; ++v) {
    if (!takes(a, v, wide)) continue;
    const F8sShape& s = kF8sShapes[v];
    const double wgs = (double)cdiv(a.M, s.rows) * (double)cdiv(a.N, s.cols);
    const double slots = (double)cus * s.per_cu;
    const double full = (double)(int64_t)(wgs / slots), rest = wgs - full * slots;
    const float n = (float)cdiv(cdiv(a.K, kF8Block), s.parts) * (wide ? s.wide : 1.0f);
    const float t = (float)full * (s.start + s.step_full * n) +
                    (rest > 0 ? s.start + (rest > slots / 2 ? s.step_full : s.step) * n : 0.0f);
    if (best == 0 || t < least) {
      best = v;
      least = t;
    }
  }
  return best;
}

}  // namespace

extern "C" {

int gemm_f8s_quantize(const gemm_f8s_quantize_args* args, void* stream) {
  if (!args) return GEMM_ERR_NULL;
  const auto [X, ldx_r, ldx_k, R, K, data, ldd, scales, lds_r, lds_k, fmt, fmt8, block_rows] = *args;
  if (!X || !data || !scales) return GEMM_ERR_NULL;
  if (R <= 0 || K <= 0 || K > kMaxK) return GEMM_ERR_SHAPE;
  if (fmt < GEMM_FMT_F16 || fmt > GEMM_FMT_F32 || fmt8 < 0 || fmt8 > 1 || (block_rows != 1 && block_rows != 128))
    return GEMM_ERR_OPTS;
  if (ldx_r <= 0 || ldx_k <= 0 || lds_r <= 0 || lds_k <= 0) return GEMM_ERR_STRIDE;
  if (ldd < K) return GEMM_ERR_LDC;
  const int64_t kb = cdiv(K, kF8Block), sr = cdiv(R, block_rows);
  Range rx, rd, rs;
  if (!byte_view(X, R, K, ldx_r, ldx_k, elem_size(fmt), &rx) || !byte_rows(data, R, ldd, K, &rd) ||
      !byte_view(scales, sr, kb, lds_r, lds_k, 4, &rs))
    return GEMM_ERR_SHAPE;
  if (!apart(sr, kb, lds_r, lds_k)) return GEMM_ERR_LDC;
  if ((uintptr_t)scales & 3u) return GEMM_ERR_LAYOUT;
  if (overlap(rx, rd) || overlap(rx, rs) || overlap(rd, rs)) return GEMM_ERR_ALIAS;

  F8QuantArgs a{X, ldx_r, ldx_k, R, K, (uint8_t*)data, ldd, scales, lds_r, lds_k, 1, {}};
  const bool tiles = block_rows == 128 || (ldx_k != 1 && K > 1);
  int64_t grid;
  if (tiles) {
    a.segs = kb;
    if (__builtin_mul_overflow(kb, cdiv(R, kF8Block), &grid)) return GEMM_ERR_SHAPE;
  } else {
    // Dense rows of whole blocks are one long row.
    if (K % kF8Block == 0 && ldx_r == K && ldd == K && lds_k == 1 && lds_r == kb) {
      a.R = 1;
      a.K = R * K;
    }
    grid = cdiv(wave_items(a.R, 16 * cdiv(a.K, kF8Block), &a.segs, &a.few), 4);
  }
  if (grid > kMaxWide) return GEMM_ERR_SHAPE;
  const bool along_k = ldx_k == 1 || K == 1;
  // Past the caches: 32768 x 7168 bfloat16 111 us instead of 125, square blocks 122
  // instead of 130, blocks along the columns 138 instead of 154.
  const bool once = (double)R * (double)K * (double)(elem_size(fmt) + 1) > kOnceBytes;
  const void* fn = fmt8 == 0 ? quant_fn<F8_E4M3>(fmt, tiles, block_rows == 128, along_k, a.few.rows > 0, once)
                             : quant_fn<F8_E5M2>(fmt, tiles, block_rows == 128, along_k, a.few.rows > 0, once);
  return run(fn, wide_grid(grid), 256, &a, (hipStream_t)stream);
}

int gemm_f8s(const gemm_f8s_args* p, void* stream) {
  if (!p) return GEMM_ERR_NULL;
  const gemm_f8s_args& q = *p;
  const int64_t M = q.M, N = q.N, K = q.K;
  if (!q.A || !q.SA || !q.B || !q.SB || !q.C) return GEMM_ERR_NULL;
  if (M <= 0 || N <= 0 || K <= 0 || K > kMaxK) return GEMM_ERR_SHAPE;
  if (q.fmt_a < 0 || q.fmt_a > 1 || q.fmt_b < 0 || q.fmt_b > 1 || (q.b_block_rows != 1 && q.b_block_rows != 128) ||
      q.fmt_c < GEMM_FMT_F16 || q.fmt_c > GEMM_FMT_F32 || q.variant < 0 || q.variant >= kF8sVariants)
    return GEMM_ERR_OPTS;
  if (q.lda <= 0 || q.ldb <= 0 || q.lsa_m <= 0 || q.lsa_k <= 0 || q.lsb_n <= 0 || q.lsb_k <= 0) return GEMM_ERR_STRIDE;
  if ((M > 1 && q.lda < K) || (N > 1 && q.ldb < K)) return GEMM_ERR_STRIDE;
  if (q.ldc < N) return GEMM_ERR_LDC;
  const int64_t kb = cdiv(K, kF8Block), nb = cdiv(N, q.b_block_rows);
  Range ra, rsa, rb, rsb, rc;
  if (!byte_rows(q.A, M, q.lda, K, &ra) || !byte_rows(q.B, N, q.ldb, K, &rb) ||
      !byte_view(q.SA, M, kb, q.lsa_m, q.lsa_k, 4, &rsa) || !byte_view(q.SB, nb, kb, q.lsb_n, q.lsb_k, 4, &rsb) ||
      !byte_view(q.C, M, N, q.ldc, 1, elem_size(q.fmt_c), &rc))
    return GEMM_ERR_SHAPE;
  if (((uintptr_t)q.A & 15u) || (M > 1 && q.lda % 16 != 0) || ((uintptr_t)q.B & 15u) || (N > 1 && q.ldb % 16 != 0) ||
      (M > 1 && (q.lda > kMaxPitch || q.lsa_m > kMaxScalePitch)) || (N > 1 && q.ldb > kMaxPitch) || (nb > 1 && q.lsb_n > kMaxScalePitch) ||
      ((uintptr_t)q.SA & 3u) || ((uintptr_t)q.SB & 3u) || ((uintptr_t)q.C % elem_size(q.fmt_c)))
    return GEMM_ERR_LAYOUT;
  if (overlap(rc, ra) || overlap(rc, rsa) || overlap(rc, rb) || overlap(rc, rsb)) return GEMM_ERR_ALIAS;
  F8sArgs a{};
  a.A = (const char*)q.A;
  a.lda = M > 1 ? q.lda : 0;
  a.SA = q.SA;
  a.sa_m = M > 1 ? q.lsa_m : 0;
  a.sa_k = q.lsa_k;
  a.B = (const char*)q.B;
  a.ldb = N > 1 ? q.ldb : 0;
  a.SB = q.SB;
  a.sb_n = nb > 1 ? q.lsb_n : 0;
  a.sb_k = q.lsb_k;
  a.C = q.C;
  a.ldc = q.ldc;
  a.M = M;
  a.N = N;
  a.K = K;
  a.out = q.fmt_c;
  a.shift = q.b_block_rows == 128 ? 7 : 0;
  a.panel = 8;   // 32768 x 2048 x 7168 by 256x256: 410 us, 443 with 4, 439 with 16
  const bool wide = q.fmt_c == GEMM_FMT_F32;
  int variant = q.variant;
  if (variant == GEMM_F8S_AUTO) {
    int cus = 0;
    const int rc = device_cus(&cus);
    if (rc) return rc;
    variant = plan(a, wide, cus);
    if (variant == GEMM_F8S_AUTO) return GEMM_ERR_SHAPE;
  } else if (!takes(a, variant, wide)) {
    return GEMM_ERR_OPTS;
  }
  const F8sShape& s = kF8sShapes[variant];
  a.GM = cdiv(M, s.rows);
  a.GN = cdiv(N, s.cols);
  const dim3 grid = s.parts > 1 ? dim3((unsigned)a.GN, (unsigned)a.GM) : dim3((unsigned)(a.GM * a.GN));
  return run(product_fn(q.fmt_a, q.fmt_b, variant, a.shift == 0, wide, q.fmt_c), grid, s.threads, &a, (hipStream_t)stream);
}

}  // extern "C"
