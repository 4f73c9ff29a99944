// Host side of include/gemm_moe.h: validation and the two launches of a
// mixture-of-experts layer for a few tokens.  Everything is checked before
// the first HIP call, so on any error nothing is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_moe.h"
#include "host_util.hpp"
#include "moe_kernel.hpp"

using namespace gemmf16;

static_assert(kMoeTokens == GEMM_MOE_MAX_TOKENS && kMoeExperts == GEMM_MOE_MAX_EXPERTS &&
                  kMoeTopK == GEMM_MOE_MAX_TOP_K,
              "bounds of the header");

namespace {

constexpr int64_t kMaxH = INT64_C(1) << 26, kMaxI = INT64_C(1) << 20;
// The kernels reach the rows of an expert's W1, of 32 rows of W2 and of all
// tokens by 32-bit offsets beside a 64-bit address.
constexpr int64_t kMaxOffset = (INT64_C(1) << 32) - (INT64_C(1) << 16);

struct Layout {
  int64_t act_row, act_part, tab_e, tab_p, sums, bytes;
};

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

bool sizes_ok(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  return T >= 1 && T <= kMoeTokens && E >= 1 && E <= kMoeExperts && k >= 1 && k <= kMoeTopK && k <= E &&
         H >= 1 && H <= kMaxH && I >= 1 && I <= kMaxI;
}

// Workgroups that may share a strip of 32 columns of Y: as many as the compute
// units have room for, at most 8.
int32_t max_splits(int64_t H, int64_t cus) {
  int32_t p = 1;
  while (p < 8 && 2 * p * cdiv(H, 32) <= cus) p *= 2;
  return p;
}
constexpr int64_t kCus = 256;   // of the whole device; a part of it splits less

Layout layout(int64_t T, int64_t k, int64_t H, int64_t I) {
  Layout l;
  l.act_row = 2 * cdiv(I, 8) * 8;
  l.act_part = up256(T * k * l.act_row);
  l.tab_e = 2 * l.act_part;
  l.tab_p = l.tab_e + up256(4 * T * k);
  l.sums = l.tab_p + up256(4 * T * k);
  const int64_t splits = max_splits(H, kCus);
  l.bytes = l.sums + (splits > 1 ? up256(4 * splits * T * cdiv(H, 32) * 32) : 0);
  return l;
}

struct Range {
  uintptr_t lo, hi;
};

// Bytes of a [G][R] stack of rows of row_bytes bytes (strides in bytes).
bool stack(const void* p, int64_t G, int64_t sg, int64_t R, int64_t sr, int64_t row_bytes, Range* out) {
  int64_t a, b;
  if (__builtin_mul_overflow(G - 1, sg, &a) || __builtin_mul_overflow(R - 1, sr, &b) ||
      __builtin_add_overflow(a, b, &a) || __builtin_add_overflow(a, row_bytes, &a) || a > INT64_MAX / 2)
    return false;
  out->lo = (uintptr_t)p;
  out->hi = out->lo + (uintptr_t)a;
  return out->hi >= out->lo;
}

// Shapes of the two kernels: strips of I (NI) or of columns of Y (NS) per wave,
// chunks per group (UC), waves per SIMD that the registers are limited to
// (WPS).  Measured per kernel (us; bf16, H 7168, I 2048, top 8 of 64 experts;
// before loads covered whole lines, which takes 6% off the 16-bit ones; up |
// down):
//   1 token, 16-bit    UC 2: 84, UC 4: 131 with the registers of WPS 4
//                      | NS 2 UC 2: 39, NS 1 UC 4: 47, NS 4 UC 2: 52
//   64 tokens, 16-bit  UC 2: 637, UC 4: 642 | NS 2 UC 2: 332, NS 1 UC 4: 386
//   16 tokens, MX4     NI 2 UC 2: 199, NI 1 UC 2: 221, NI 2 UC 1: 265
//                      | few: NS 2 UC 2: 110, NS 2 UC 1: 126, NS 1 UC 1: 138,
//                      NS 1 UC 2: 161; not few: NS 2 UC 1: 152, NS 1 UC 1: 200
//   64 tokens, MX4     NI 1 UC 2: 270, NI 1 UC 1: 331, NI 2 UC 1: spills
//   H 2048, I 768, 4 tokens, 16-bit: down NS 1 UC 4 11.5 (few: 9.9), NS 2 UC 2
//   14.7: where NS 2 leaves compute units without work, NS 1, or NS 2 with the
//   sums split (see launch_kernels)
// "few" is the down kernel's form for experts with few tokens each.  It pays
// while most have four or fewer, measured by the mean over all experts, T k / E
// (16 tokens; few | not, us): MX4 2: 110 | 152, 3: 68 | 105, 4: 75 | 100, 6: 45
// | 51, 8: 52 | 53, 16: 44 | 36; 16-bit 2: 261 | 263, 3: 155 | 150, 6: 100 | 83.
// With more than 16 tokens its registers and LDS cost more than it saves (64
// tokens, mean 8, 16-bit: 439 | 325).
template <int WF, int MT>
struct Shape {
  static constexpr int NI = 1, UP_UC = 2, UP_WPS = MT == 1 ? 4 : 2;
  static constexpr int UC_NS1 = MT == 1 ? 4 : 2, UC_NS2 = 2, FEW_UC_NS2 = 2, DOWN_WPS = MT == 1 ? 4 : 2;
  static constexpr int FEW_MEAN = 2, SPLIT_K = 32 * 40;
};
template <int MT>
struct Shape<SW_MX4, MT> {
  static constexpr int NI = MT == 1 ? 2 : 1, UP_UC = 2, UP_WPS = 2;
  static constexpr int UC_NS1 = 1, UC_NS2 = 1, FEW_UC_NS2 = 2, DOWN_WPS = 2;
  static constexpr int FEW_MEAN = 4, SPLIT_K = 128 * 12;
};

template <int WF, int DT, int MT, int NS, int UC, bool FEW, bool ONCE>
int launch_down(MoeArgs& a, hipStream_t s) {
  void* p[] = {&a};
  if (hipLaunchKernel((const void*)moe_down_kernel<WF, DT, MT, NS, UC, Shape<WF, MT>::DOWN_WPS, FEW, ONCE>,
                      dim3((unsigned)cdiv(a.H, 16 * NS), (unsigned)a.splits), dim3(64 * kMoeWaves), p, 0, s) !=
      hipSuccess)
    return GEMM_ERR_HIP;
  if (a.splits > 1 && hipLaunchKernel((const void*)moe_sum_kernel<DT>,
                                      dim3((unsigned)cdiv(a.H, 4 * 256), (unsigned)a.T), dim3(256), p, 0, s) != hipSuccess)
    return GEMM_ERR_HIP;
  return GEMM_OK;
}

// The last cache holds 256 MiB: weights that half of it can keep from call to
// call are read through it (7 experts of 9.4 MB, 4 tokens: the layer 22 to 23.4 us,
// past it 24.4).
constexpr int64_t kCached = INT64_C(128) << 20;

template <int WF, int DT, int MT, bool ONCE>
int launch_kernels(MoeArgs& a, int cus, hipStream_t s) {
  using P = Shape<WF, MT>;
  // Parts of H per strip of I: as few as give the device six waves per compute
  // unit (at most min(E, T top_k) experts are in use).
  const int64_t strips = cdiv(a.I, 16 * P::NI) * std::min(a.E, a.T * a.k);
  a.parts = 1;
  while (a.parts < kMoeWaves && strips * a.parts < (int64_t)6 * cus) a.parts *= 2;
  void* p[] = {&a};
  const dim3 up((unsigned)cdiv(a.I, 16 * P::NI * (kMoeWaves / a.parts)), (unsigned)(a.by_pair ? a.T * a.k : a.E));
  if (hipLaunchKernel((const void*)moe_up_kernel<WF, DT, MT, P::NI, P::UP_UC, P::UP_WPS, ONCE>, up, dim3(64 * kMoeWaves),
                      p, 0, s) != hipSuccess)
    return GEMM_ERR_HIP;
  // Two strips of columns a wave where they give three quarters of the compute
  // units a workgroup.  With fewer columns the (expert, group) sequence of a strip
  // is split over workgroups that fill the device, and a third kernel adds their
  // sums, if a wave's share without is long enough to pay for that, SPLIT_K of I
  // (us, one strip and no split | two and split): H 2048, I 768, 48 tokens, 128
  // experts, 16-bit: 166 | 76, MX4 123 | 54; 16 tokens, 64 experts, MX4: 47 | 23,
  // H 4096: 48 | 31; H 1000, I 600, 10 tokens, 30 experts: 16-bit 20 | 16, MX4
  // 19.1 | 16.4; H 2048, I 768, 4 tokens, top 2 of 16: 10.0 | 11.5; H 1400, I
  // 500, 8 experts: 18.1 | 19.1.  (The strip's last workgroup adding the sums
  // instead of a kernel: 120 instead of 76, its fences write the L2 back.)
  bool two = 4 * cdiv(a.H, 32) >= 3 * (int64_t)cus;
  a.splits = 1;
  if (!two && std::min<int64_t>(a.E, a.T * a.k) * a.I >= (int64_t)P::SPLIT_K * kMoeWaves) {
    a.splits = max_splits(a.H, std::min<int64_t>(cus, kCus));
    two = a.splits > 1;
  }
  if constexpr (MT == 1) {
    if (a.T <= 4 || a.T * a.k <= P::FEW_MEAN * a.E)
      return two ? launch_down<WF, DT, MT, 2, P::FEW_UC_NS2, true, ONCE>(a, s)
                 : launch_down<WF, DT, MT, 1, P::UC_NS1, true, false>(a, s);
  }
  return two ? launch_down<WF, DT, MT, 2, P::UC_NS2, false, ONCE>(a, s)
             : launch_down<WF, DT, MT, 1, P::UC_NS1, false, false>(a, s);
}

template <int WF, int DT>
int launch_layer(MoeArgs& a, int cus, hipStream_t s) {
  if constexpr (WF != SW_MX4) {
    if (std::min<int64_t>(a.E, a.T * a.k) * 6 * a.H * a.I > kCached)
      return a.T <= 16 ? launch_kernels<WF, DT, 1, true>(a, cus, s) : launch_kernels<WF, DT, 4, true>(a, cus, s);
  }
  return a.T <= 16 ? launch_kernels<WF, DT, 1, false>(a, cus, s) : launch_kernels<WF, DT, 4, false>(a, cus, s);
}

}  // namespace

extern "C" {

size_t gemm_moe_workspace_bytes(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I) {
  return sizes_ok(T, E, top_k, H, I) ? (size_t)layout(T, top_k, H, I).bytes : 0;
}

int gemm_moe(const gemm_moe_args* g, void* stream, void* workspace, size_t workspace_bytes) {
  if (!g || !g->X || !g->logits || !g->W1 || !g->W2 || !g->Y || (g->mx4 == 1 && (!g->S1 || !g->S2)))
    return GEMM_ERR_NULL;
  if (!sizes_ok(g->T, g->E, g->top_k, g->H, g->I)) return GEMM_ERR_SHAPE;
  if ((g->fmt != GEMM_FMT_F16 && g->fmt != GEMM_FMT_BF16) || g->fmt_logits < GEMM_FMT_F16 ||
      g->fmt_logits > GEMM_FMT_F32 || (g->mx4 != 0 && g->mx4 != 1))
    return GEMM_ERR_OPTS;
  const int64_t T = g->T, E = g->E, H = g->H, I = g->I;
  const int64_t hb = cdiv(H, kMxBlock), ib = cdiv(I, kMxBlock);
  // Row lengths and strides of the weights in bytes.
  const int64_t es = g->mx4 ? 1 : 2;
  const int64_t row1 = g->mx4 ? hb * kMxBytes : 2 * H, row2 = g->mx4 ? ib * kMxBytes : 2 * I;
  if (g->ldx <= 0 || g->ldl <= 0 || g->w1_n <= 0 || g->w2_n <= 0 || g->w1_e < 0 || g->w2_e < 0)
    return GEMM_ERR_STRIDE;
  if (g->mx4 && (g->s1_n <= 0 || g->s2_n <= 0 || g->s1_e < 0 || g->s2_e < 0 || g->w1_n < row1 || g->s1_n < hb ||
                 (H > 1 && (g->w2_n < row2 || g->s2_n < ib))))
    return GEMM_ERR_STRIDE;
  if (g->ldy < H) return GEMM_ERR_LDC;
  if (std::max({g->ldx, g->ldl, g->ldy, g->w1_n, g->w2_n, g->w1_e, g->w2_e}) > INT64_MAX / 8)
    return GEMM_ERR_SHAPE;
  const int64_t el = g->fmt_logits == GEMM_FMT_F32 ? 4 : 2;
  Range rx, rl, r1, r2, rs1{0, 0}, rs2{0, 0}, ry;
  if (!stack(g->X, 1, 0, T, 2 * g->ldx, 2 * H, &rx) || !stack(g->logits, 1, 0, T, el * g->ldl, el * E, &rl) ||
      !stack(g->W1, E, es * g->w1_e, 2 * I, es * g->w1_n, row1, &r1) ||
      !stack(g->W2, E, es * g->w2_e, H, es * g->w2_n, row2, &r2) ||
      !stack(g->Y, 1, 0, T, 2 * g->ldy, 2 * H, &ry))
    return GEMM_ERR_SHAPE;
  if (g->mx4 && (!stack(g->S1, E, g->s1_e, 2 * I, g->s1_n, hb, &rs1) ||
                 !stack(g->S2, E, g->s2_e, H, g->s2_n, ib, &rs2)))
    return GEMM_ERR_SHAPE;
  if ((T - 1) * g->ldx > kMaxOffset / 2 || es * g->w1_n > kMaxOffset / (2 * I) || es * g->w2_n > kMaxOffset / 32 ||
      (g->mx4 && (g->s1_n > kMaxOffset / (2 * I) || g->s2_n > kMaxOffset / 32)))
    return GEMM_ERR_LAYOUT;
  const Range* in[] = {&rx, &rl, &r1, &r2, &rs1, &rs2};
  for (const Range* r : in)
    if (ranges_overlap(ry.lo, ry.hi, r->lo, r->hi)) return GEMM_ERR_ALIAS;
  const Layout l = layout(T, g->top_k, H, I);

  MoeArgs a;
  a.x = (const char*)g->X;
  a.ldx = 2 * g->ldx;
  a.logits = g->logits;
  a.ldl = g->ldl;
  a.w1 = (const char*)g->W1;
  a.w2 = (const char*)g->W2;
  a.w1_e = es * g->w1_e;
  a.w1_n = es * g->w1_n;
  a.w2_e = es * g->w2_e;
  a.w2_n = es * g->w2_n;
  a.s1 = (const uint8_t*)g->S1;
  a.s2 = (const uint8_t*)g->S2;
  a.s1_e = g->s1_e;
  a.s1_n = g->s1_n;
  a.s2_e = g->s2_e;
  a.s2_n = g->s2_n;
  a.y = (uint16_t*)g->Y;
  a.ldy = g->ldy;
  a.act_row = l.act_row;
  a.act_part = l.act_part;
  a.H = H;
  a.I = I;
  a.T = (int32_t)T;
  a.E = (int32_t)E;
  a.k = g->top_k;
  a.fmt_l = g->fmt_logits;
  // Fewer pairs than experts: most experts are unused, so workgroups go by
  // pair (each finds its expert) instead of by expert.
  a.by_pair = T * g->top_k < E;
  a.renormalize = g->renormalize != 0;

  hipStream_t s = (hipStream_t)stream;
  void* ws = workspace;
  if (workspace) {
    if (workspace_bytes < (size_t)l.bytes || ((uintptr_t)workspace & 255u)) return GEMM_ERR_WORKSPACE;
    const uintptr_t w0 = (uintptr_t)workspace, w1 = w0 + (uintptr_t)l.bytes;
    for (const Range* r : in)
      if (ranges_overlap(w0, w1, r->lo, r->hi)) return GEMM_ERR_ALIAS;
    if (ranges_overlap(w0, w1, ry.lo, ry.hi)) return GEMM_ERR_ALIAS;
  }
  int cus = 0;
  int rc = device_cus(&cus);
  if (rc) return rc;
  if (!workspace && hipMallocAsync(&ws, (size_t)l.bytes, s) != hipSuccess) return GEMM_ERR_HIP;
  a.act = (char*)ws;
  a.tab_e = (int32_t*)((char*)ws + l.tab_e);
  a.tab_p = (float*)((char*)ws + l.tab_p);
  a.sums = (float*)((char*)ws + l.sums);
  a.sums_row = cdiv(H, 32) * 32;
  if (g->mx4)
    rc = g->fmt == GEMM_FMT_F16 ? launch_layer<SW_MX4, DT_F16>(a, cus, s) : launch_layer<SW_MX4, DT_BF16>(a, cus, s);
  else
    rc = g->fmt == GEMM_FMT_F16 ? launch_layer<SW_F16, DT_F16>(a, cus, s) : launch_layer<SW_BF16, DT_BF16>(a, cus, s);
  if (!workspace && hipFreeAsync(ws, s) != hipSuccess && rc == GEMM_OK) rc = GEMM_ERR_HIP;
  return rc;
}

}  // extern "C"
