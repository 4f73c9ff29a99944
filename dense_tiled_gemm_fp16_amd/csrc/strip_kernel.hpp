// Products with few rows of A (gfx950): the inner loop of the decode forms
// with [N, K] weights, 16-bit or MX FP4.
//
// With few rows the time goes to reading the weights once, so the loop is
// built around those loads: a wave owns NS strips of 16 weight rows and a
// range of K, loads the weights 16 bytes per lane straight into registers (no
// LDS: no other wave of the workgroup wants them), the loads of the next UC
// chunks in flight while this one's are multiplied, and the waves of a
// workgroup, which share the strips and split K, add their sums through LDS at
// the end.  The few rows of A come from L1/L2.
//
// The matrix instruction is 16 x 16 (k 32, or 128 for MX4 x MX4), its first
// operand the weights: lane l holds weight row l % 16 and, of each chunk, the
// k octet or block l / 16; the sums land as weight rows 4 (l / 16) + r of
// column (row of A) l % 16.  Only the order of k is free, as long as both
// operands share it:
//   16-bit weights   a chunk is 32 k; lane group g takes octet g (16 bytes).
//   MX4 weights      a chunk is 128 k, 64 bytes of a row; lane group g takes
//                    block g (16 bytes, one scale).  With a 16-bit A dword j
//                    of the block meets octet 4 g + j of the chunk in the
//                    j-th of four instructions; with an MX4 A one scaled
//                    128-k instruction takes the chunk.
//
// Weights in MX4 are widened exactly: to bfloat16 at any scale; to binary16,
// for a binary16 A, where the scale byte is in 104 .. 140 (or below 61, where
// the terms vanish next to binary16's least step whatever A holds).  Other
// scales take the chunk through bfloat16, A split exactly into two bfloat16
// parts.
//
// Rows past the end read a valid row (their sums are never stored); k past K
// enters as zero on both sides.
#pragma once

#include "mx4_common.hpp"

namespace gemmf16 {

enum StripW { SW_F16 = 0, SW_BF16 = 1, SW_MX4 = 2 };
// A operand: 16-bit rows, two 16-bit parts whose sum is the value (rows xp
// bytes apart), or MX4 rows.
enum StripX { SX_F16 = 0, SX_BF16 = 1, SX_F16P = 2, SX_BF16P = 3, SX_MX4 = 4 };

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
template <class T>
__device__ __forceinline__ T as8(u32x4 v) {
  return __builtin_bit_cast(T, v);
}

// Elements k .. k+7 of a 16-bit row, zero from K on.
__device__ __forceinline__ u32x4 load8_tail(const char* row, int64_t k, int64_t K) {
  if (k + 8 <= K) return load16(row + 2 * k);
  const int64_t n = K - k;
  return load_partial8((const uint16_t*)row + (n > 0 ? k : 0), 1, n > 0 ? (int)n : 0);
}

// binary16 -> two bfloat16 parts, exactly: 11 significant bits as 8 + 3.
__device__ __forceinline__ void split_bf16(f16x8 x, bf16x8& hi, bf16x8& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = (float)x[i];
    hi[i] = (__bf16)f;
    const float r = f - (float)hi[i];
    lo[i] = (__bf16)(r == r ? r : 0.0f);   // an infinity leaves no rest
  }
}

template <int WF, int XF, int NS_, int MT_, int UC_>
struct Strip {
  static constexpr int NS = NS_, MT = MT_, UC = UC_;
  static constexpr bool W4 = WF == SW_MX4, X4 = XF == SX_MX4;
  static constexpr int PL = (XF == SX_F16P || XF == SX_BF16P) ? 2 : 1;
  static constexpr int CK = W4 ? 128 : 32;                  // k per chunk
  static constexpr int XV = X4 ? 1 : (W4 ? 4 : 1);          // 16-byte A loads per chunk and part
  static_assert(W4 || !X4, "MX4 A takes MX4 weights");

  const char* w[NS];        // this lane's weight rows
  const uint8_t* ws[NS];    // their scales (MX4)
  const char* x[MT];        // this lane's rows of A
  const uint8_t* xs[MT];    // their scales (MX4)
  int64_t xp;               // bytes to the second part's rows

  struct WBuf {
    u32x4 v[UC][NS];
    uint32_t s[UC][NS];
  };

  static __device__ __forceinline__ int64_t chunks(int64_t K) { return (K + CK - 1) / CK; }

  // Weights of chunks c .. c+UC-1, none from `end` on (uniform bounds).
  __device__ __forceinline__ void load_w(WBuf& b, int64_t c, int64_t end, int64_t K, int g) const {
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      const int64_t cc = c + u;
      if (cc < end) {
        const bool full = (cc + 1) * CK <= K;
        if constexpr (W4) {
          const int64_t blk = 4 * cc + g;
          const bool ok = full || blk * 32 < K;
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            b.v[u][s] = ok ? load16(w[s] + blk * 16) : zero4();
            b.s[u][s] = ok ? ws[s][blk] : 127u;
          }
        } else {
          const int64_t k = cc * 32 + 8 * g;
#pragma unroll
          for (int s = 0; s < NS; ++s)
            b.v[u][s] = full ? load16(w[s] + 2 * k) : load8_tail(w[s], k, K);
        }
      }
    }
  }

  // Sums over chunks [c0, c1).
  __device__ __forceinline__ void run(f32x4 (&acc)[NS][MT], int64_t c0, int64_t c1, int64_t K, int lane) const {
    const int g = lane >> 4;
    WBuf cur, nxt;
    load_w(cur, c0, c1, K, g);
    for (int64_t c = c0; c < c1; c += UC) {
      u32x4 xv[UC][MT][PL][XV];
      uint32_t xsc[UC][MT];
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        const int64_t cc = c + u;
        if (cc < c1) {
          const bool full = (cc + 1) * CK <= K;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            if constexpr (X4) {
              const int64_t blk = 4 * cc + g;
              const int64_t left = K - blk * 32;
              const bool ok = full || left > 0;
              xv[u][t][0][0] = ok ? load16(x[t] + blk * 16) : zero4();
              if (!full && left < 32) xv[u][t][0][0] = mask_codes(xv[u][t][0][0], (int)left);
              xsc[u][t] = ok ? xs[t][blk] : 127u;
            } else {
#pragma unroll
              for (int p = 0; p < PL; ++p)
#pragma unroll
                for (int j = 0; j < XV; ++j) {
                  const int64_t k = cc * CK + g * (8 * XV) + 8 * j;
                  const char* row = x[t] + p * xp;
                  xv[u][t][p][j] = full ? load16(row + 2 * k) : load8_tail(row, k, K);
                }
            }
          }
        }
      }
      load_w(nxt, c + UC, c1, K, g);
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        if (c + u < c1) {
          if constexpr (X4) {
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                const u32x4 a = cur.v[u][s], b = xv[u][t][0][0];
                const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
                const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
                acc[s][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    av, bv, acc[s][t], 4, 4, 0, (int)cur.s[u][s], 0, (int)xsc[u][t]);
              }
          } else if constexpr (W4) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              const float sc = scale_f32(cur.s[u][s]);
              if constexpr (XF == SX_F16) {
                const uint32_t b = cur.s[u][s];
                if (__any(b > 140 || (b > 60 && b < 104))) {
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const bf16x8 wf = mx4_to_bf16(cur.v[u][s][j], sc);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                      bf16x8 hi, lo;
                      split_bf16(as8<f16x8>(xv[u][t][0][j]), hi, lo);
                      acc[s][t] = mfma16(wf, lo, acc[s][t]);
                      acc[s][t] = mfma16(wf, hi, acc[s][t]);
                    }
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const f16x8 wf = mx4_to_f16(cur.v[u][s][j], sc);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                      acc[s][t] = mfma16(wf, as8<f16x8>(xv[u][t][0][j]), acc[s][t]);
                  }
                }
              } else {
                static_assert(XF != SX_F16P, "MX4 weights take bfloat16 parts");
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const bf16x8 wf = mx4_to_bf16(cur.v[u][s][j], sc);
#pragma unroll
                  for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int p = PL - 1; p >= 0; --p)
                      acc[s][t] = mfma16(wf, as8<bf16x8>(xv[u][t][p][j]), acc[s][t]);
                }
              }
            }
          } else {
            using V = std::conditional_t<WF == SW_F16, f16x8, bf16x8>;
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
              for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int p = PL - 1; p >= 0; --p)
                  acc[s][t] = mfma16(as8<V>(cur.v[u][s]), as8<V>(xv[u][t][p][0]), acc[s][t]);
          }
        }
      }
      cur = nxt;
    }
  }
};

// Sum of a tile's partial sums over the NW waves, in wave order: part holds
// [NW][TILES][64 lanes] float4.
template <int NW, int TILES>
__device__ __forceinline__ f32x4 sum_waves(const f32x4* part, int tile, int lane) {
  f32x4 s = part[tile * 64 + lane];
#pragma unroll
  for (int w = 1; w < NW; ++w) {
    const f32x4 v = part[(w * TILES + tile) * 64 + lane];
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] += v[r];
  }
  return s;
}

constexpr int kStripWaves = 8;

struct StripArgs {
  const char* a;
  int64_t lda;            // bytes
  const uint8_t* as;
  int64_t ldas;
  const char* b;
  int64_t ldb;            // bytes
  const uint8_t* bs;
  int64_t ldbs;
  uint16_t* c;
  int64_t ldc, M, N, K;
};

// C[m,n] = sum_k A[m,k] B[n,k] with MX4 B: workgroup -> (16 NS columns of C,
// 16 MT rows), its waves the ranges of K.
template <int XF, int DT, int NS, int MT, int UC>
__global__ __launch_bounds__(64 * kStripWaves) void mx4_strip_kernel(StripArgs a) {
  using S = Strip<SW_MX4, XF, NS, MT, UC>;
  constexpr int TILES = NS * MT;
  static_assert(TILES <= kStripWaves, "one thread per float4 of the tiles");
  __shared__ f32x4 part[kStripWaves * TILES * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NS), m0 = (int64_t)blockIdx.y * (16 * MT);
  S s;
  s.xp = 0;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    int64_t n = n0 + 16 * i + (lane & 15);
    if (n >= a.N) n = a.N - 1;
    s.w[i] = a.b + n * a.ldb;
    s.ws[i] = a.bs + n * a.ldbs;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    int64_t m = m0 + 16 * t + (lane & 15);
    if (m >= a.M) m = a.M - 1;
    s.x[t] = a.a + m * a.lda;
    s.xs[t] = a.as + m * a.ldas;
  }
  f32x4 acc[NS][MT];
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t nc = S::chunks(a.K);
  s.run(acc, nc * wave / kStripWaves, nc * (wave + 1) / kStripWaves, a.K, lane);
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) part[(wave * TILES + i * MT + t) * 64 + lane] = acc[i][t];
  __syncthreads();
  if (wave < TILES) {
    const f32x4 v = sum_waves<kStripWaves, TILES>(part, wave, lane);
    const int i = wave / MT, t = wave % MT;
    const int64_t m = m0 + 16 * t + (lane & 15), n = n0 + 16 * i + 4 * (lane >> 4);
    if (m < a.M && n < a.N) {
      uint16_t* c = a.c + m * a.ldc + n;
      uint16_t h[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) h[r] = cvt_out<DT>(v[r]);
      if (n + 4 <= a.N) {
        __builtin_memcpy(c, h, 8);
      } else {
        for (int r = 0; r < 4 && n + r < a.N; ++r) c[r] = h[r];
      }
    }
  }
}

}  // namespace gemmf16
