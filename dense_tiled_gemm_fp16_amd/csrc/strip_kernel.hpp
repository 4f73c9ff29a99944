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

// Wait states after matrix instructions, tied to their sums.  The compiler
// counts the cycles a result needs before other instructions may read it within
// a basic block, but leaves them out where the reader, often only a register
// move, is the first of the next block: a group's sums pass through here
// before any branch.  (16 states; the longest instruction here needs 12.)
__device__ __forceinline__ void settle(f32x4 (&a)[1]) { asm volatile("s_nop 15" : "+v"(a[0])); }
__device__ __forceinline__ void settle(f32x4 (&a)[2]) { asm volatile("s_nop 15" : "+v"(a[0]), "+v"(a[1])); }
__device__ __forceinline__ void settle(f32x4 (&a)[4]) {
  asm volatile("s_nop 15" : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]));
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

// NS strips of 16 weight rows x MT tiles of 16 rows of A, UC chunks at a time.
// `g` is the lane's group, lane / 16.
template <int WF, int XF, int NS_, int MT_, int UC_>
struct Strip {
  static constexpr int NS = NS_, MT = MT_, UC = UC_;
  static constexpr bool W4 = WF == SW_MX4, X4 = XF == SX_MX4;
  static constexpr int PL = (XF == SX_F16P || XF == SX_BF16P) ? 2 : 1;
  static constexpr int CK = W4 ? 128 : 32;                  // k per chunk
  static constexpr int XV = X4 ? 1 : (W4 ? 4 : 1);          // 16-byte A loads per chunk and part
  static_assert(W4 || !X4, "MX4 A takes MX4 weights");

  struct WPtr {
    const char* w[NS];        // this lane's weight rows
    const uint8_t* s[NS];     // their scales (MX4)
  };
  struct XPtr {
    const char* x[MT];        // this lane's rows of A
    const uint8_t* s[MT];     // their scales (MX4)
    int64_t part;             // bytes to the second part's rows
  };
  struct WBuf {
    u32x4 v[UC][NS];
    uint32_t s[UC][NS];
  };
  struct XBuf {
    u32x4 v[UC][MT][PL][XV];
    uint32_t s[UC][MT];
  };

  static __device__ __forceinline__ int64_t chunks(int64_t K) { return (K + CK - 1) / CK; }

  static __device__ __forceinline__ void clear(f32x4 (&acc)[NS][MT]) {
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[s][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // A whole group: all its chunks exist and end by K.
  static __device__ __forceinline__ bool whole(int64_t c, int64_t end, int64_t K) {
    return c + UC <= end && (c + UC) * CK <= K;
  }

  // Weights of chunks c .. c+UC-1, zeros from `end` on (uniform bounds).
  static __device__ __forceinline__ void load_w(WBuf& b, const WPtr& p, int64_t c, int64_t end, int64_t K,
                                                int g) {
    if (whole(c, end, K)) {
#pragma unroll
      for (int u = 0; u < UC; ++u)
#pragma unroll
        for (int s = 0; s < NS; ++s) b.v[u][s] = load16(p.w[s] + (c + u) * 64 + 16 * g);
      if constexpr (W4) {
        // One load of the group's 4 UC scales, the lane's picked by shifts.
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          uint32_t d[UC];
          __builtin_memcpy(d, p.s[s] + 4 * c, 4 * UC);
#pragma unroll
          for (int u = 0; u < UC; ++u) b.s[u][s] = (d[u] >> (8 * g)) & 255u;
        }
      }
      return;
    }
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      const int64_t cc = c + u;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        b.v[u][s] = zero4();
        b.s[u][s] = 127u;
      }
      if (cc < end) {
        if constexpr (W4) {
          const int64_t blk = 4 * cc + g;
          if (blk * 32 < K) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              b.v[u][s] = load16(p.w[s] + blk * 16);
              b.s[u][s] = p.s[s][blk];
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < NS; ++s) b.v[u][s] = load8_tail(p.w[s], cc * 32 + 8 * g, K);
        }
      }
    }
  }

  // The same chunks of A, of all tiles or (one) the first alone.
  static __device__ __forceinline__ void load_x(XBuf& b, const XPtr& p, int64_t c, int64_t end, int64_t K, int g,
                                                bool one) {
    const bool all = whole(c, end, K);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if (t > 0 && one) continue;
      if (all) {
        if constexpr (X4) {
          uint32_t d[UC];
          __builtin_memcpy(d, p.s[t] + 4 * c, 4 * UC);
#pragma unroll
          for (int u = 0; u < UC; ++u) {
            b.v[u][t][0][0] = load16(p.x[t] + (c + u) * 64 + 16 * g);
            b.s[u][t] = (d[u] >> (8 * g)) & 255u;
          }
        } else {
#pragma unroll
          for (int u = 0; u < UC; ++u)
#pragma unroll
            for (int q = 0; q < PL; ++q)
#pragma unroll
              for (int j = 0; j < XV; ++j)
                b.v[u][t][q][j] = load16(p.x[t] + q * p.part + (c + u) * (2 * CK) + g * (16 * XV) + 16 * j);
        }
        continue;
      }
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        const int64_t cc = c + u;
#pragma unroll
        for (int q = 0; q < PL; ++q)
#pragma unroll
          for (int j = 0; j < XV; ++j) b.v[u][t][q][j] = zero4();
        b.s[u][t] = 127u;
        if (cc < end) {
          if constexpr (X4) {
            const int64_t blk = 4 * cc + g, left = K - blk * 32;
            if (left > 0) {
              b.v[u][t][0][0] = mask_codes(load16(p.x[t] + blk * 16), left < 32 ? (int)left : 32);
              b.s[u][t] = p.s[t][blk];
            }
          } else {
#pragma unroll
            for (int q = 0; q < PL; ++q)
#pragma unroll
              for (int j = 0; j < XV; ++j)
                b.v[u][t][q][j] = load8_tail(p.x[t] + q * p.part, cc * CK + g * (8 * XV) + 8 * j, K);
          }
        }
      }
    }
  }

  // Products of a group, T tiles of A, without a branch between the matrix
  // instructions (see settle).
  template <int T, bool WIDE>
  static __device__ __forceinline__ void mma_tiles(f32x4 (&acc)[NS][MT], const WBuf& wb, const XBuf& xb) {
#pragma unroll
    for (int u = 0; u < UC; ++u) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if constexpr (X4) {
          const u32x4 a = wb.v[u][s];
          const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
#pragma unroll
          for (int t = 0; t < T; ++t) {
            const u32x4 b = xb.v[u][t][0][0];
            const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
            acc[s][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[s][t], 4, 4, 0,
                                                                         (int)wb.s[u][s], 0, (int)xb.s[u][t]);
          }
        } else if constexpr (W4) {
          const float sc = scale_f32(wb.s[u][s]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (XF == SX_F16 && !WIDE) {
              const f16x8 wf = mx4_to_f16(wb.v[u][s][j], sc);
#pragma unroll
              for (int t = 0; t < T; ++t) acc[s][t] = mfma16(wf, as8<f16x8>(xb.v[u][t][0][j]), acc[s][t]);
            } else {
              static_assert(XF != SX_F16P, "MX4 weights take bfloat16 parts");
              const bf16x8 wf = mx4_to_bf16(wb.v[u][s][j], sc);
#pragma unroll
              for (int t = 0; t < T; ++t) {
                if constexpr (XF == SX_F16) {
                  bf16x8 hi, lo;
                  split_bf16(as8<f16x8>(xb.v[u][t][0][j]), hi, lo);
                  acc[s][t] = mfma16(wf, lo, acc[s][t]);
                  acc[s][t] = mfma16(wf, hi, acc[s][t]);
                  __builtin_amdgcn_sched_barrier(0);   // one split's registers at a time
                } else {
#pragma unroll
                  for (int q = PL - 1; q >= 0; --q)
                    acc[s][t] = mfma16(wf, as8<bf16x8>(xb.v[u][t][q][j]), acc[s][t]);
                }
              }
            }
          }
        } else {
          using V = std::conditional_t<WF == SW_F16, f16x8, bf16x8>;
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int q = PL - 1; q >= 0; --q)
              acc[s][t] = mfma16(as8<V>(wb.v[u][s]), as8<V>(xb.v[u][t][q][0]), acc[s][t]);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) settle(acc[s]);
  }

  static __device__ __forceinline__ void mma(f32x4 (&acc)[NS][MT], const WBuf& wb, const XBuf& xb, bool one) {
    bool wide = false;
    if constexpr (W4 && XF == SX_F16) {   // scales that binary16 does not hold
#pragma unroll
      for (int u = 0; u < UC; ++u)
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const uint32_t b = wb.s[u][s];
          wide = wide || b > 140 || (b > 60 && b < 104);
        }
      wide = __any(wide);
    }
    if (W4 && XF == SX_F16 && wide) {
      if (MT > 1 && one)
        mma_tiles<1, true>(acc, wb, xb);
      else
        mma_tiles<MT, true>(acc, wb, xb);
    } else {
      if (MT > 1 && one)
        mma_tiles<1, false>(acc, wb, xb);
      else
        mma_tiles<MT, false>(acc, wb, xb);
    }
  }

  // Sums over chunks [c0, c1); `one`: only the first tile of A is in use.
  static __device__ __forceinline__ void run(f32x4 (&acc)[NS][MT], const WPtr& wp, const XPtr& xp, int64_t c0,
                                             int64_t c1, int64_t K, int g, bool one) {
    WBuf cur, nxt;
    XBuf x;
    load_w(cur, wp, c0, c1, K, g);
    for (int64_t c = c0; c < c1; c += UC) {
      load_x(x, xp, c, c1, K, g, one);
      if (c + UC < c1) load_w(nxt, wp, c + UC, c1, K, g);
      mma(acc, cur, x, one);
      cur = nxt;
    }
  }
};

// Sum of a tile's partial sums over n waves, in wave order; part points at the
// first wave's tile, waves `stride` float4s apart.
__device__ __forceinline__ f32x4 sum_waves(const f32x4* part, int stride, int n, int lane) {
  f32x4 s = part[lane];
  for (int w = 1; w < n; ++w) {
    const f32x4 v = part[w * stride + lane];
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] += v[r];
  }
  return s;
}

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
// 16 MT rows), its NW waves the ranges of K.
template <int XF, int DT, int NS, int MT, int UC, int NW>
__global__ __launch_bounds__(64 * NW, MT < 2 ? 4 : 2) void mx4_strip_kernel(StripArgs a) {
  using S = Strip<SW_MX4, XF, NS, MT, UC>;
  constexpr int TILES = NS * MT;
  __shared__ f32x4 part[NW * TILES * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NS), m0 = (int64_t)blockIdx.y * (16 * MT);
  typename S::WPtr w;
  typename S::XPtr x;
  x.part = 0;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    int64_t n = n0 + 16 * i + (lane & 15);
    if (n >= a.N) n = a.N - 1;
    w.w[i] = a.b + n * a.ldb;
    w.s[i] = a.bs + n * a.ldbs;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    int64_t m = m0 + 16 * t + (lane & 15);
    if (m >= a.M) m = a.M - 1;
    x.x[t] = a.a + m * a.lda;
    x.s[t] = a.as + m * a.ldas;
  }
  f32x4 acc[NS][MT];
  S::clear(acc);
  const int64_t nc = S::chunks(a.K);
  S::run(acc, w, x, nc * wave / NW, nc * (wave + 1) / NW, a.K, lane >> 4, a.M - m0 <= 16);
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) part[(wave * TILES + i * MT + t) * 64 + lane] = acc[i][t];
  __syncthreads();
  for (int tile = wave; tile < TILES; tile += NW) {
    const f32x4 v = sum_waves(part + tile * 64, TILES * 64, NW, lane);
    const int i = tile / MT, t = tile % MT;
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
