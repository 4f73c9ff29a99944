// Host side of include/gemm_mx4.h: argument validation and launches of the
// MX FP4 quantiser, its inverse and the products with MX4 weights.  Everything
// is checked before the first HIP call, so on any error nothing is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_mx4.h"
#include "host_launch.hpp"
#include "mx4_convert.hpp"
#include "mx4_tile_kernel.hpp"
#include "strip_kernel.hpp"

using namespace gemmf16;

namespace {

int64_t elem_size(int32_t fmt) { return fmt == GEMM_FMT_F32 ? 4 : 2; }

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

// How rows of octs octets are dealt to wave items; returns their number.
int64_t wave_items(int64_t rows, int64_t octs, int64_t* segs, Short* few) {
  *segs = cdiv(octs, kSlots);
  *few = Short{};
  if (*segs > 1 || rows == 1) return rows * *segs;
  *few = Short{(int32_t)octs, (int32_t)(kSlots / octs), (int32_t)(65536 / octs + 1)};
  return cdiv(rows, few->rows);
}
template <int FMT>
const void* rows_kernel(const Short& few) {
  return few.rows ? (const void*)quantize_rows_kernel<FMT, true> : (const void*)quantize_rows_kernel<FMT, false>;
}
template <int FMT>
const void* back_kernel(const Short& few) {
  return few.rows ? (const void*)dequantize_kernel<FMT, true> : (const void*)dequantize_kernel<FMT, false>;
}

// K up to 2^36, as the 16-bit tiles: chunk counters stay far inside int64.
constexpr int64_t kMaxK = INT64_C(1) << 36;

template <int XF, int DT, int NS, int MT, int UC, int NW, bool FEW = false>
int launch_strip(const StripArgs& a, hipStream_t s) {
  const int64_t gx = cdiv(a.N, 16 * NS), gy = cdiv(a.M, 16 * MT);
  StripArgs copy = a;
  return run((const void*)mx4_strip_kernel<XF, DT, NS, MT, UC, NW, FEW>, dim3((unsigned)gx, (unsigned)gy), 64 * NW,
             &copy, s);
}

// The strip kernel's lanes reach 64 rows of A and 32 rows of B by 32-bit
// offsets: row strides of at most 2^26 bytes.
constexpr int64_t kMaxStripLd = INT64_C(1) << 26;
bool strip_takes(const StripArgs& a) {
  return a.lda <= kMaxStripLd && a.ldas <= kMaxStripLd && a.ldb <= kMaxStripLd && a.ldbs <= kMaxStripLd;
}

// How many strips of 16 columns a wave takes, and how many rows: as many as
// leave three quarters of the compute units a workgroup, since each further
// strip shares the A that the wave turns through LDS and each further tile of
// rows the weights.  Measured (us per kernel in a graph of 50; NS = strips,
// rows x N x K):
//   16-bit A   up to 4 rows (FEW), bfloat16 unless said: 1 x 2048 x 7168: 4.4,
//              without FEW 5.4; binary16: 5.3, 6.1; 1 x 7168 x 2048 binary16:
//              NS 1 3.9, without 4.7; NS 2 4.0, 4.2; 1 x 28672 x 4096 binary16:
//              NS 1 17.2, 19.6; NS 2 15.4, 16.6
//              16 x 7168 x 2048: NS 1 5.1, NS 2 4.2
//              32 x 7168 x 7168, 32 rows a wave: NS 1 15.7, 2 11.8, 4 15.8
//              64 x 7168 x 7168, 32 rows: NS 1 28.0, 2 20.5, 4 16.5; 64 rows,
//              NS 2: 20.1
//   MX4 A      16 x 7168 x 2048: NS 1 3.9, NS 2 3.6
//              64 rows a wave, 333 x 1061 x 2050: NS 2 7.1, 4 9.1;
//              512 x 2048 x 7168: NS 2 22.0, 4 18.2; 1024 x 2048 x 7168:
//              NS 4 34.2, with four waves instead of eight 31.9
template <int XF, int DT>
int launch_strip_m(const StripArgs& a, hipStream_t s) {
  if (!strip_takes(a)) return GEMM_ERR_LAYOUT;
  // The grid: fewer than 2^32 work items along x, 65535 workgroups along y.
  if (a.N > (INT64_C(1) << 27) || cdiv(a.M, XF == SX_MX4 ? 64 : 32) > 65535) return GEMM_ERR_SHAPE;
  int cus = 0;
  const int rc = device_cus(&cus);
  if (rc) return rc;
  const int64_t enough = 3 * (int64_t)cus / 4;
  if constexpr (XF != SX_MX4) {
    if (a.M <= 4)
      return cdiv(a.N, 32) >= enough ? launch_strip<XF, DT, 2, 1, 1, 8, true>(a, s)
                                     : launch_strip<XF, DT, 1, 1, 1, 8, true>(a, s);
  }
  if (a.M <= 16) {
    if (cdiv(a.N, 32) >= enough) return launch_strip<XF, DT, 2, 1, 1, 8>(a, s);
    return launch_strip<XF, DT, 1, 1, XF == SX_MX4 ? 2 : 1, 8>(a, s);
  }
  if constexpr (XF == SX_MX4) {
    const int64_t wgs = cdiv(a.N, 64) * cdiv(a.M, 64);
    if (wgs < enough) return launch_strip<XF, DT, 2, 4, 1, 8>(a, s);
    if (4 * wgs <= 5 * (int64_t)cus) return launch_strip<XF, DT, 4, 4, 1, 8>(a, s);
    return launch_strip<XF, DT, 4, 4, 1, 4>(a, s);
  } else {
    const int64_t m = cdiv(a.M, 32);
    if (cdiv(a.N, 64) * m >= enough) return launch_strip<XF, DT, 4, 2, 1, 8>(a, s);
    if (cdiv(a.N, 32) * m >= enough) return launch_strip<XF, DT, 2, 2, 1, 8>(a, s);
    return launch_strip<XF, DT, 1, 2, 1, 8>(a, s);
  }
}

// The tile kernel's plan: its scale arrays, transposed, are the workspace; the
// grids of the kernel that transposes them (gx, gy) and of the tiles.
struct TilePlan {
  int64_t steps, sa_rows, sb_rows, gx, gy, grid;
};

// False for more workgroups than a launch takes.
bool tile_plan(int64_t M, int64_t N, int64_t K, TilePlan* p) {
  p->steps = cdiv(K, 128);
  p->sa_rows = cdiv(M, Mx4Cfg::BM) * Mx4Cfg::BM;
  p->sb_rows = cdiv(N, Mx4Cfg::BN) * Mx4Cfg::BN;
  p->gx = cdiv(std::max(p->sa_rows, p->sb_rows), 64);
  p->gy = cdiv(p->steps, 16);
  return !__builtin_mul_overflow(p->sa_rows / Mx4Cfg::BM, p->sb_rows / Mx4Cfg::BN, &p->grid) &&
         fits_x(p->grid, Mx4Cfg::NT) && fits_x(p->gx, 256) && p->gy <= 65535;
}

// 256 x 256 tiles from 48 of them on (1024 x 2048 x 7168, 32 tiles: 41.3 us
// against 31.9 by strips; 2048^3, 64 tiles: 17.5 against 21.0; 1024 x 4096 x
// 4096, 64: 26.2 against 36.2), unless most of each tile would be empty.  Lane
// offsets span 255 rows in 32 bits.
bool takes_tile(int64_t M, int64_t N, int64_t K) {
  return M > 128 && N > 128 && (double)cdiv(M, Mx4Cfg::BM) * (double)cdiv(N, Mx4Cfg::BN) >= 48 && K <= (INT64_C(1) << 24);
}
constexpr int64_t kMaxTileLd = INT64_C(1) << 24;

template <int DT>
int launch_tile(const StripArgs& a, const TilePlan& p, void* ws, hipStream_t s) {
  uint32_t* sa = (uint32_t*)ws;
  uint32_t* sb = sa + p.steps * p.sa_rows;
  Mx4ScaleArgs q{{a.as, a.bs}, {a.ldas, a.ldbs}, {a.M, a.N}, {p.sa_rows, p.sb_rows}, {sa, sb},
                 cdiv(a.K, kMxBlock), p.steps};
  Mx4TileArgs t{};
  t.k.A = (const uint16_t*)a.a;
  t.k.lda_m = a.lda;
  t.k.B = (const uint16_t*)a.b;
  t.k.ldb_n = a.ldb;
  t.k.C = a.c;
  t.k.ldc = a.ldc;
  t.k.M = a.M;
  t.k.N = a.N;
  t.k.K = a.K;
  t.k.GM = cdiv(a.M, Mx4Cfg::BM);
  t.k.GN = cdiv(a.N, Mx4Cfg::BN);
  t.k.panel = 8;   // 32768 x 2048 x 7168, one run: 228 us, 236 with 4, 235 with 16; within 1% on squares
  t.sa = sa;
  t.sa_rows = p.sa_rows;
  t.sb = sb;
  t.sb_rows = p.sb_rows;
  const int rc = run((const void*)mx4_scales_kernel, dim3((unsigned)p.gx, (unsigned)p.gy, 2), 256, &q, s);
  if (rc) return rc;
  return run((const void*)mx4_tile_kernel<DT>, dim3((unsigned)p.grid), Mx4Cfg::NT, &t, s);
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

  QuantArgs a{X, ldx_g, ldx_r, ldx_k, G, R, K, (uint8_t*)data, (uint8_t*)scales, Kb, 1, {}};
  if (G > 1 && ldx_g == R * ldx_r) {   // one stack of rows
    a.G = 1;
    a.R = rows;
  }
  int64_t grid;
  int threads = 256;
  const void* fn;
  if (ldx_k == 1) {
    // Dense rows of whole blocks are one long row.
    if (K % kMxBlock == 0 && ldx_r == K && a.G == 1) {
      a.R = 1;
      a.K = rows * K;
      a.Kb = rows * Kb;
    }
    grid = cdiv(wave_items(a.G * a.R, 4 * a.Kb, &a.segs, &a.few), 4);
    fn = fmt == GEMM_FMT_F16    ? rows_kernel<MX_F16>(a.few)
         : fmt == GEMM_FMT_BF16 ? rows_kernel<MX_BF16>(a.few)
                                : rows_kernel<MX_F32>(a.few);
  } else {
    threads = 64 * kColBlocks;
    a.segs = cdiv(Kb, kColBlocks);
    grid = cdiv(rows, 64) * a.segs;
    fn = fmt == GEMM_FMT_F16    ? (const void*)quantize_columns_kernel<MX_F16>
         : fmt == GEMM_FMT_BF16 ? (const void*)quantize_columns_kernel<MX_BF16>
                                : (const void*)quantize_columns_kernel<MX_F32>;
  }
  if (grid > kMaxWide) return GEMM_ERR_SHAPE;
  return run(fn, wide_grid(grid), threads, &a, (hipStream_t)stream);
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

  DequantArgs a{(const uint8_t*)data, ldd, (const uint8_t*)scales, lds, R, K, Y, ldy, 1, {}};
  const int64_t kb = cdiv(K, kMxBlock);
  if (K % kMxBlock == 0 && ldy == K && ldd == kb * kMxBytes && lds == kb) {   // one long row
    a.R = 1;
    a.K = R * K;
  }
  const int64_t grid = cdiv(wave_items(a.R, cdiv(a.K, 8), &a.segs, &a.few), 4);
  if (grid > kMaxWide) return GEMM_ERR_SHAPE;
  const void* fn = fmt == GEMM_FMT_F16    ? back_kernel<MX_F16>(a.few)
                   : fmt == GEMM_FMT_BF16 ? back_kernel<MX_BF16>(a.few)
                                          : back_kernel<MX_F32>(a.few);
  return run(fn, wide_grid(grid), 256, &a, (hipStream_t)stream);
}

size_t gemm_mx4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > INT64_MAX / 8 || N > INT64_MAX / 8 || !takes_tile(M, N, K)) return 0;
  const int64_t rows = cdiv(M, 256) * 256 + cdiv(N, 256) * 256;
  int64_t bytes;
  if (__builtin_mul_overflow(4 * cdiv(K, 128), rows, &bytes)) return 0;
  return (size_t)bytes;
}

int gemm_mx4(const void* A, int64_t lda, const void* SA, int64_t ldsa, const void* B, int64_t ldb,
             const void* SB, int64_t ldsb, void* C, int32_t fmt_c, int64_t ldc, int64_t M, int64_t N,
             int64_t K, void* stream, void* workspace, size_t workspace_bytes) {
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
  if (M == 1) lda = ldsa = 0;   // a single row has no next one
  if (N == 1) ldb = ldsb = 0;
  const StripArgs a{(const char*)A, lda, (const uint8_t*)SA, ldsa, (const char*)B, ldb, (const uint8_t*)SB,
                    ldsb, (uint16_t*)C, ldc, M, N, K};
  hipStream_t s = (hipStream_t)stream;
  const bool f16 = fmt_c == GEMM_FMT_F16;
  if (!takes_tile(M, N, K) || lda > kMaxTileLd || ldb > kMaxTileLd)
    return f16 ? launch_strip_m<SX_MX4, DT_F16>(a, s) : launch_strip_m<SX_MX4, DT_BF16>(a, s);
  const size_t need = gemm_mx4_workspace_bytes(M, N, K);
  TilePlan plan;
  if (need == 0 || !tile_plan(M, N, K, &plan)) return GEMM_ERR_SHAPE;
  void* ws = workspace;
  if (workspace) {
    if (workspace_bytes < need || ((uintptr_t)workspace & 255u)) return GEMM_ERR_WORKSPACE;
    const Range rw{(uintptr_t)workspace, (uintptr_t)workspace + need};
    if (overlap(rw, ra) || overlap(rw, rsa) || overlap(rw, rb) || overlap(rw, rsb) || overlap(rw, rc_))
      return GEMM_ERR_ALIAS;
  } else if (hipMallocAsync(&ws, need, s) != hipSuccess) {
    return GEMM_ERR_HIP;
  }
  rc = f16 ? launch_tile<DT_F16>(a, plan, ws, s) : launch_tile<DT_BF16>(a, plan, ws, s);
  if (!workspace && hipFreeAsync(ws, s) != hipSuccess && rc == GEMM_OK) rc = GEMM_ERR_HIP;
  return rc;
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
  if (M == 1) lda = 0;   // a single row has no next one
  if (N == 1) ldb = ldsb = 0;
  const StripArgs a{(const char*)A, 2 * lda, nullptr, 0, (const char*)B, ldb, (const uint8_t*)SB, ldsb,
                    (uint16_t*)C, ldc, M, N, K};
  return fmt == GEMM_FMT_F16 ? launch_strip_m<SX_F16, DT_F16>(a, (hipStream_t)stream)
                             : launch_strip_m<SX_BF16, DT_BF16>(a, (hipStream_t)stream);
}

}  // extern "C"
