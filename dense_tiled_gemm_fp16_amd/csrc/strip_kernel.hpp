// Products with few rows of A (gfx950): the inner loop of the decode forms
// with [N, K] weights, 16-bit or MX FP4.
//
// With few rows the time goes to reading the weights once, so the loop is
// built around those loads: a wave owns NS strips of 16 weight rows and a
// range of K and keeps the weights of two groups of UC chunks (64 bytes per
// row each) in flight beside the group that it multiplies; waves that share
// strips and split K add their sums through LDS at the end.  The few rows of A
// come from L2 the same way, one group ahead.  Loads return in order, so a
// group's A is issued before the weights of the group after it: waiting for
// the former then leaves the latter in flight.
//
// The matrix instruction is 16 x 16 (k 32, or 128 for MX4 x MX4), its first
// operand the weights: lane l holds weight row l % 16 and k octet or block
// l / 16; the sums land as weight rows 4 (l / 16) + r of column (row of A)
// l % 16.  Loaded in that arrangement, every four neighbouring lanes touch four
// rows, and the address unit takes 64 cycles for a 1 KiB load instruction; four
// lanes on the 64 bytes of one row take 16 (both measured).  So neighbouring
// lanes load neighbouring 16-byte pieces of a row (of the group's 64 UC bytes of
// weights, of a chunk's 64 bytes of A), and the pieces change lanes through a
// part of LDS that belongs to the wave: written and read in the wave's own
// order, without barriers.  The slot of a row's piece is XORed with bits of the
// row, which keeps both sides free of bank conflicts.
//
// Measured per kernel (medians of a kernel trace): one token, H 7168, I 2048, 8
// experts in bfloat16 6.3 and 5.5 TB/s (75 and 43 us), 64 tokens, 64 experts 6.4
// and 5.8; plain reads of the same bytes 6.4; as products with MX4 weights, in a
// graph, 1 x 2048 x 7168 5.5 us and 16 x 7168 x 2048 4.4 us, of which some 2.5 are
// a launch and the sum over the waves.
//
// Only the order of k is free, as long as both operands share it:
//   16-bit weights   a chunk is 32 k; lane group g takes octet g.
//   MX4 weights      a chunk is 128 k; lane group g takes block g (16 bytes,
//                    one scale).  With a 16-bit A, dword j of the block meets
//                    octet 4 g + j of the chunk in the j-th of four
//                    instructions; with an MX4 A one scaled 128-k instruction
//                    takes the chunk.
//
// Weights in MX4 are widened exactly: to bfloat16 at any scale (values of 2^128
// and more, which the quantiser does not give, become infinite there); to binary16,
// for a binary16 A, where the scale byte is in 104 .. 140.  Other scales take
// the chunk through bfloat16, A split exactly into two bfloat16 parts; all but
// 0, the scale of a block of zeros: whatever nonzero codes it has (up to 2^-124)
// vanish next to binary16's least step.  Binary16 weights that meet an A in
// bfloat16 parts are split exactly into two such parts too.
//
// Rows past the end read a valid row (their sums are never stored); k past K
// enters as zero on both sides.
#pragma once

#include "dma_a128_kernel.hpp"
#include "mx4_common.hpp"

namespace gemmf16 {

enum StripW { SW_F16 = 0, SW_BF16 = 1, SW_MX4 = 2 };
// A operand: 16-bit rows, two bfloat16 parts whose sum is the value (rows xp
// bytes apart), or MX4 rows.
enum StripX { SX_F16 = 0, SX_BF16 = 1, SX_BF16P = 2, SX_MX4 = 3 };

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

// Weights are read once.  Where a load's lanes cover whole lines and the last
// cache could not keep them until the next call they need not stay in any
// (ONCE): the layer's first kernel, 16-bit, 64 tokens 593 us instead of 632, 16
// tokens 554 instead of 584, its second at 16 tokens 250 instead of 263.  Half
// lines (UC 1) are fetched twice that way: 719 instead of 590.  No gain for MX4
// (16 tokens 201 | 199, 2 tokens 57 | 50) or UC 4 (13 | 12).
template <bool ONCE>
__device__ __forceinline__ u32x4 load_weights(const void* p) {
  typedef u32x4 Any __attribute__((aligned(1)));
  if constexpr (ONCE)
    return __builtin_nontemporal_load((const GEMM_GLOBAL Any*)p);
  else
    return load16(p);
}

// The first n of the eight 16-bit elements at p, the others zero.
__device__ __forceinline__ u32x4 load8_rest(const char* p, int64_t n) {
  if (n >= 8) return load16(p);
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = e < n ? (uint32_t)gload<uint16_t>(p + 2 * e) : 0u;
  return u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
}

// Wait states after matrix instructions, tied to their sums.  The compiler
// counts the cycles a result needs before other instructions may read it within
// a basic block, but has left them out where the reader, often only a register
// move, was the first of the next block: a group's sums pass through here
// before any branch.  (16 states; the longest instruction here needs 12.)
template <int N, int MT>
__device__ __forceinline__ void settle(f32x4 (&a)[N][MT], int t) {
  if constexpr (N == 1) {
    asm volatile("s_nop 15" : "+v"(a[0][t]));
  } else if constexpr (N == 2) {
    asm volatile("s_nop 15" : "+v"(a[0][t]), "+v"(a[1][t]));
  } else {
    static_assert(N == 4, "strips of a wave");
    asm volatile("s_nop 15" : "+v"(a[0][t]), "+v"(a[1][t]), "+v"(a[2][t]), "+v"(a[3][t]));
  }
}

// binary16 -> two bfloat16 parts, exactly: 11 significant bits as 8 + 3.  An
// infinity leaves no rest, or with FINITE (inputs that are) a NaN.
template <bool FINITE>
__device__ __forceinline__ void split_bf16(f16x8 x, bf16x8& hi, bf16x8& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = (float)x[i];
    hi[i] = (__bf16)f;
    const float r = f - (float)hi[i];
    lo[i] = (__bf16)(FINITE || r == r ? r : 0.0f);
  }
}

// Order of one wave's LDS accesses: the hardware keeps it, the compiler has to
// be told that lanes read what other lanes wrote.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// NS strips of 16 weight rows x MT tiles of 16 rows of A, UC chunks at a time.
// XT: tiles of A that run ahead; the others are fetched when they are needed
// (see more_tiles).  FEW: of the first tile only the first FR rows run ahead,
// one row's pieces of the whole group side by side in a load (a quarter of the
// loads and LDS writes), the others are fetched when there are any.
template <int WF, int XF, int NS_, int MT_, int UC_, int XT = MT_, bool FEW_ = false, bool ONCE = false>
struct Strip {
  static constexpr int NS = NS_, MT = MT_, UC = UC_;
  static constexpr bool W4 = WF == SW_MX4, X4 = XF == SX_MX4;
  static constexpr int PL = XF == SX_BF16P ? 2 : 1;
  static constexpr int CK = W4 ? 128 : 32;                  // k per chunk
  static constexpr int XV = X4 ? 1 : (W4 ? 4 : 1);          // 64-byte pieces of A per chunk, row and part
  static_assert(W4 || !X4, "MX4 A takes MX4 weights");
  static_assert(XT == 1 || XT == MT_, "one tile ahead, or all");
  static_assert(!ONCE || UC == 2, "a row's piece of a load is a line");
  static constexpr bool FEW = FEW_;
  // FEW: pieces of 16 bytes per row of A in a group, rows per load, rows and
  // loads that run ahead.
  static constexpr int PR = 4 * UC * PL * XV, RPL = 64 / PR, FR = RPL > 4 ? RPL : 4, FL = FR / RPL;
  static_assert(!FEW || (XT == 1 && !X4 && PR >= 8 && PR <= 64), "a load takes whole rows");
  // FEW with two parts: a tile is 8 rows, columns c and c + 8 of the products
  // are the first and the second part of row c (to be added in the end), so the
  // parts share an instruction.
  static constexpr bool PACK = FEW && PL == 2;
  static constexpr int PM = PACK ? 1 : PL, TR = PACK ? 8 : 16;   // products per octet; rows of a tile
  // A wave's LDS: the group's weights, one chunk of one part of A (FEW: 16 rows
  // of the whole group), scales.
  static constexpr int X_AT = UC * NS * 1024, S_AT = X_AT + (FEW ? TR * 16 * PR : XV * 1024),
                       XS_AT = S_AT + (W4 ? NS * 16 * UC * 4 : 0);
  static constexpr int LDS = XS_AT + (X4 ? 16 * UC * 4 : 0);

  // A group's weights: WP pieces of 16 bytes a row, WR rows a load, so that the
  // lanes of one load cover whole lines.  In LDS a row's pieces lie side by side.
  static constexpr int WP = 4 * UC, WR = 64 / WP;
  static __device__ __forceinline__ int w_row(int i, int lane) { return i * WR + lane / WP; }
  static __device__ __forceinline__ int w_slot(int r, int piece) {
    return r * (16 * WP) + ((piece ^ (UC == 1 ? fa(r) : r & 7)) << 4);
  }

  // A uniform address and the lane's 32-bit offset beside it, so that moving
  // along K or to another expert is scalar arithmetic.
  struct WPtr {
    const char* w;            // the strips' first row
    const uint8_t* s;         // its scales (MX4)
  };
  struct WOff {
    uint32_t w[NS][UC];       // row w_row(i, lane) of each strip, piece lane % WP
    uint32_t s[NS];           // scales of row lane for lanes 0 .. 15, of row 0 for the others (MX4)
  };
  struct XPtr {
    const char* x;            // uniform, as for the weights
    const uint8_t* s;
    uint32_t xo;              // the lane's row
    uint32_t so;              // scales of row lane % 16 of its tile (MX4 A)
  };

  // Offsets of strips that start `stride` rows apart, `rows` rows from the
  // first strip's first one on existing.
  static __device__ __forceinline__ WOff offsets(int64_t rows, int64_t stride, int64_t ld, int64_t lds, int lane) {
    WOff o;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
#pragma unroll
      for (int j = 0; j < UC; ++j) {
        int64_t r = i * stride + w_row(j, lane);
        if (r >= rows) r = rows - 1;
        o.w[i][j] = (uint32_t)(r * ld) + 16 * (lane % WP);
      }
      int64_t q = i * stride + (lane < 16 ? lane : 0);
      if (q >= rows) q = rows - 1;
      o.s[i] = (uint32_t)(q * lds);
    }
    return o;
  }

  struct WRegs {
    u32x4 w[UC][NS];
    uint32_t s[NS][UC];
  };
  struct XRegs {
    u32x4 x[UC][PL][XV];
    uint32_t xs[UC];
  };
  struct XFew {
    u32x4 x[FL];
  };
  using XAhead = std::conditional_t<FEW, XFew, XRegs>;

  static __device__ __forceinline__ int64_t chunks(int64_t K) { return (K + CK - 1) / CK; }

  static __device__ __forceinline__ void clear(f32x4 (&acc)[NS][MT]) {
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[s][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // Whole groups of a row of K, and whether chunks are left behind them.
  static __device__ __forceinline__ int64_t groups(int64_t K) { return K / (UC * CK); }
  static __device__ __forceinline__ bool rest(int64_t K) { return K % (UC * CK) != 0; }

  // The loads of a whole group, chunks c .. c+UC-1, are straight-line code: a
  // branch around them would make the compiler join their registers with
  // others behind it, by moves that wait for the loads at once.
  static __device__ __forceinline__ void load_w(WRegs& b, const WPtr& p, const WOff& o, int64_t c) {
    const char* w = uniform_ptr(p.w + c * 64);
#pragma unroll
    for (int u = 0; u < UC; ++u)
#pragma unroll
      for (int s = 0; s < NS; ++s) b.w[u][s] = load_weights<ONCE>(w + o.w[s][u]);
    if constexpr (W4) {
      const char* sp = uniform_ptr((const char*)p.s + 4 * c);
#pragma unroll
      for (int s = 0; s < NS; ++s) load_dwords(b.s[s], sp + o.s[s]);
    }
  }
  static __device__ __forceinline__ void load_x(XRegs& b, const XPtr& p, int64_t xpart, int64_t c, int lane) {
    const char* x = uniform_ptr(p.x + c * (64 * XV));
    const uint32_t xo = p.xo + 16 * (lane & 3);
#pragma unroll
    for (int u = 0; u < UC; ++u)
#pragma unroll
      for (int q = 0; q < PL; ++q)
#pragma unroll
        for (int j = 0; j < XV; ++j) b.x[u][q][j] = load16(x + q * xpart + xo + u * (64 * XV) + 64 * j);
    if constexpr (X4) load_dwords(b.xs, uniform_ptr((const char*)p.s + 4 * c) + p.so);
  }

  // The last, partial group of a row: chunks c .. , zeros past K.
  static __device__ __forceinline__ void load_w_rest(WRegs& b, const WPtr& p, const WOff& o, int64_t c, int64_t K,
                                                     int lane) {
    const int64_t k0 = c * CK + (W4 ? 32 : 8) * (lane % WP);   // of the lane's piece
#pragma unroll
    for (int u = 0; u < UC; ++u)
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const char* w = p.w + c * 64 + o.w[s][u];
        if constexpr (W4) {
          // a code behind K may stand for more than bfloat16 holds, and an
          // infinity times the zero that it meets would be NaN
          b.w[u][s] = k0 < K ? mask_codes(load16(w), K - k0 < 32 ? (int)(K - k0) : 32) : zero4();
          b.s[s][u] = scales_rest(p.s + 4 * (c + u) + o.s[s], c + u, K);
        } else {
          b.w[u][s] = load8_rest(w, K - k0);
        }
      }
  }
  static __device__ __forceinline__ void load_x_rest(XRegs& b, const XPtr& p, int64_t xpart, int64_t c, int64_t K,
                                                     int lane) {
    const int piece = lane & 3;
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      const int64_t cc = c + u;
      if constexpr (X4) {
        const int64_t left = K - (4 * cc + piece) * 32;
        b.x[u][0][0] = left > 0 ? mask_codes(load16(p.x + cc * 64 + p.xo + 16 * piece), left < 32 ? (int)left : 32) : zero4();
        b.xs[u] = scales_rest(p.s + 4 * cc + p.so, cc, K);
      } else {
#pragma unroll
        for (int q = 0; q < PL; ++q)
#pragma unroll
          for (int j = 0; j < XV; ++j)
            b.x[u][q][j] = load8_rest(p.x + cc * (64 * XV) + q * xpart + p.xo + 64 * j + 16 * piece,
                                      K - (cc * CK + 32 * j + 8 * piece));
      }
    }
  }

  // The four scales of chunk c at p, 2^0 past K.
  static __device__ __forceinline__ uint32_t scales_rest(const uint8_t* p, int64_t c, int64_t K) {
    uint32_t d = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) d |= ((4 * c + i) * 32 < K ? (uint32_t)gload<uint8_t>(p + i) : 127u) << (8 * i);
    return d;
  }

  // A group's weights and scales into the wave's LDS.
  static __device__ __forceinline__ void stage_w(char* lds, const WRegs& b, int lane) {
    wave_order();
#pragma unroll
    for (int u = 0; u < UC; ++u)
#pragma unroll
      for (int s = 0; s < NS; ++s)
        *(u32x4*)(lds + s * (1024 * UC) + w_slot(w_row(u, lane), lane % WP)) = b.w[u][s];
    if constexpr (W4) {
      if (lane < 16) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int u = 0; u < UC; ++u) *(uint32_t*)(lds + S_AT + ((s * 16 + lane) * UC + u) * 4) = b.s[s][u];
      }
    }
  }

  // Chunk u, part q of A through the wave's LDS: this lane's octets.
  static __device__ __forceinline__ void turn_x(char* lds, const XRegs& b, int u, int q, u32x4 (&f)[XV], int lane) {
    wave_order();
    const int wr = lane >> 2, at = wr * 64 + (((lane & 3) ^ fa(wr)) << 4);
#pragma unroll
    for (int j = 0; j < XV; ++j) *(u32x4*)(lds + X_AT + j * 1024 + at) = b.x[u][q][j];
    wave_order();
    const int r = lane & 15, g = lane >> 4;
    if constexpr (XV == 1) {
      f[0] = *(const u32x4*)(lds + X_AT + r * 64 + ((g ^ fa(r)) << 4));
    } else {
#pragma unroll
      for (int j = 0; j < XV; ++j) f[j] = *(const u32x4*)(lds + X_AT + g * 1024 + r * 64 + ((j ^ fa(r)) << 4));
    }
  }

  // A tile's octets of the whole group.
  struct XFrags {
    u32x4 f[UC][PM][XV];
    uint32_t s[UC];
  };
  static __device__ __forceinline__ void turn(XFrags& f, char* lds, const XRegs& b, int lane) {
    if constexpr (X4) {
      wave_order();
      if (lane < 16) {
#pragma unroll
        for (int u = 0; u < UC; ++u) *(uint32_t*)(lds + XS_AT + (lane * UC + u) * 4) = b.xs[u];
      }
    }
#pragma unroll
    for (int u = 0; u < UC; ++u) {
#pragma unroll
      for (int q = 0; q < PL; ++q) turn_x(lds, b, u, q, f.f[u][q], lane);
      if constexpr (X4) f.s[u] = *(const uint32_t*)(lds + XS_AT + ((lane & 15) * UC + u) * 4) >> (8 * (lane >> 4));
    }
  }

  // FEW: lane l takes piece l % PR of row l / PR of a load; pieces of a row count
  // chunk, part, octet.  In LDS a row's pieces lie side by side, piece p of row
  // r in slot p ^ (r % 8): both sides free of bank conflicts.
  template <bool REST, class Cursor>
  static __device__ __forceinline__ void load_few(XFew& b, const Cursor& cc, int row, int64_t xpart, int64_t K,
                                                  int lane) {
    const int piece = lane % PR, w = piece % (4 * XV), u = piece / (4 * XV * PL), q = piece / (4 * XV) % PL;
    const uint32_t off = (uint32_t)(q * xpart) + u * (64 * XV) + 16 * w;
#pragma unroll
    for (int i = 0; i < FL; ++i) {
      const XPtr p = cc.x(row + i * RPL + lane / PR);
      const char* x = uniform_ptr(p.x + cc.c() * (64 * XV));
      if constexpr (REST)
        b.x[i] = load8_rest(x + (p.xo + off), K - ((cc.c() + u) * CK + 8 * w));
      else
        b.x[i] = load16(x + (p.xo + off));
    }
  }
  static __device__ __forceinline__ void store_few(char* lds, const XFew& b, int row, int lane) {
#pragma unroll
    for (int i = 0; i < FL; ++i) {
      const int r = row + i * RPL + lane / PR;
      *(u32x4*)(lds + X_AT + r * (16 * PR) + ((lane % PR ^ (r & 7)) << 4)) = b.x[i];
    }
  }
  // Rows `row` .. of tile t, fetched now.
  template <bool REST, class Cursor>
  static __device__ __forceinline__ void fetch_few(char* lds, const Cursor& cc, int t, int row, int64_t xpart,
                                                   int64_t K, int lane) {
    const int rows = cc.rows() - TR * t;
    for (; row < TR && row < rows; row += FR) {
      XFew b;
      load_few<REST>(b, cc, TR * t + row, xpart, K, lane);
      store_few(lds, b, row, lane);
    }
  }
  static __device__ __forceinline__ void read_few(XFrags& f, const char* lds, int lane) {
    wave_order();
    const int r = lane & (TR - 1), g = lane >> 4, part = PACK ? (lane & 15) / TR : 0;
#pragma unroll
    for (int u = 0; u < UC; ++u)
#pragma unroll
      for (int q = 0; q < PM; ++q)
#pragma unroll
        for (int j = 0; j < XV; ++j) {
          const int p = (u * PL + q + part) * (4 * XV) + (XV == 1 ? g : 4 * g + j);
          f.f[u][q][j] = *(const u32x4*)(lds + X_AT + r * (16 * PR) + ((p ^ (r & 7)) << 4));
        }
  }

  // Products of the staged group with tile T of A, no branch between the
  // matrix instructions (see settle), the strips in turn so that neighbouring
  // instructions do not wait for each other's sums.
  template <int T, bool WIDE>
  static __device__ __forceinline__ void mma_tile(f32x4 (&acc)[NS][MT], const char* lds, const XFrags& x, int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      u32x4 w[NS];
      uint32_t sb[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        w[s] = *(const u32x4*)(lds + s * (1024 * UC) + w_slot(r, 4 * u + g));
        if constexpr (W4) sb[s] = (*(const uint32_t*)(lds + S_AT + ((s * 16 + r) * UC + u) * 4) >> (8 * g)) & 255u;
      }
      if constexpr (X4) {
        const u32x4 b = x.f[u][0][0];
        const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const i32x8 av = {(int)w[s][0], (int)w[s][1], (int)w[s][2], (int)w[s][3], 0, 0, 0, 0};
          acc[s][T] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[s][T], 4, 4, 0, (int)sb[s], 0,
                                                                       (int)x.s[u]);
        }
      } else if constexpr (W4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (XF == SX_F16 && WIDE) {
            bf16x8 hi, lo;
            split_bf16<false>(as8<f16x8>(x.f[u][0][j]), hi, lo);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              const bf16x8 wf = mx4_to_bf16(w[s][j], scale_f32(sb[s]));
              acc[s][T] = mfma16(wf, lo, acc[s][T]);
              acc[s][T] = mfma16(wf, hi, acc[s][T]);
            }
            __builtin_amdgcn_sched_barrier(0);   // one octet's registers at a time
          } else {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              if constexpr (XF == SX_F16) {
                acc[s][T] = mfma16(mx4_to_f16(w[s][j], scale_f32(sb[s])), as8<f16x8>(x.f[u][0][j]), acc[s][T]);
              } else {
                const bf16x8 wf = mx4_to_bf16(w[s][j], scale_f32(sb[s]));
#pragma unroll
                for (int q = PM - 1; q >= 0; --q)   // the smaller part first
                  acc[s][T] = mfma16(wf, as8<bf16x8>(x.f[u][q][j]), acc[s][T]);
              }
            }
          }
        }
      } else if constexpr (WF == SW_F16 && XF == SX_BF16P) {
        bf16x8 hi[NS], lo[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) split_bf16<true>(as8<f16x8>(w[s]), hi[s], lo[s]);
#pragma unroll
        for (int q = PM - 1; q >= 0; --q) {   // the smaller parts first
          const bf16x8 xf = as8<bf16x8>(x.f[u][q][0]);
#pragma unroll
          for (int s = 0; s < NS; ++s) acc[s][T] = mfma16(lo[s], xf, acc[s][T]);
#pragma unroll
          for (int s = 0; s < NS; ++s) acc[s][T] = mfma16(hi[s], xf, acc[s][T]);
        }
      } else {
        using V = std::conditional_t<WF == SW_F16, f16x8, bf16x8>;
#pragma unroll
        for (int q = PM - 1; q >= 0; --q)
#pragma unroll
          for (int s = 0; s < NS; ++s) acc[s][T] = mfma16(as8<V>(w[s]), as8<V>(x.f[u][q][0]), acc[s][T]);
      }
    }
    settle(acc, T);
  }

  // Some scale of the group is one that binary16 does not hold (lanes 0 .. 15
  // have them).
  static __device__ __forceinline__ bool wide(const WRegs& b, int lane) {
    bool w = false;
    if constexpr (W4 && XF == SX_F16) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int u = 0; u < UC; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = (b.s[s][u] >> (8 * i)) & 255u;
            w = w || x > 140 || (x > 0 && x < 104);
          }
      w = __any(w && lane < 16);
    }
    return w;
  }

  template <int T>
  static __device__ __forceinline__ void mma(f32x4 (&acc)[NS][MT], const char* lds, const XFrags& x, bool is_wide,
                                             int lane) {
    if (W4 && XF == SX_F16 && is_wide)
      mma_tile<T, true>(acc, lds, x, lane);
    else
      mma_tile<T, false>(acc, lds, x, lane);
  }

  template <int T>
  static __device__ __forceinline__ void mma_all(f32x4 (&acc)[NS][MT], const char* lds, const XFrags* f, bool is_wide,
                                                 int lane) {
    mma<T>(acc, lds, f[T], is_wide, lane);
    if constexpr (T + 1 < XT) mma_all<T + 1>(acc, lds, f, is_wide, lane);
  }

  // Tiles 1 .. tiles-1 of A against the staged group where only tile 0 runs
  // ahead.
  template <int T, bool REST, class Cursor>
  static __device__ __forceinline__ void more_tiles(f32x4 (&acc)[NS][MT], char* lds, const Cursor& cc, int64_t xpart,
                                                    int64_t K, bool is_wide, int lane) {
    if constexpr (T < MT && XT == 1) {
      if (TR * T < cc.rows()) {
        XFrags x;
        if constexpr (FEW) {
          wave_order();
          fetch_few<REST>(lds, cc, T, 0, xpart, K, lane);
          read_few(x, lds, lane);
        } else {
          XRegs b;
          if constexpr (REST)
            load_x_rest(b, tile(cc, T, lane), xpart, cc.c(), K, lane);
          else
            load_x(b, tile(cc, T, lane), xpart, cc.c(), lane);
          turn(x, lds, b, lane);
        }
        mma<T>(acc, lds, x, is_wide, lane);
        more_tiles<T + 1, REST>(acc, lds, cc, xpart, K, is_wide, lane);
      }
    }
  }

  // This lane's rows of tile t.
  template <class Cursor>
  static __device__ __forceinline__ XPtr tile(const Cursor& cc, int t, int lane) {
    return cc.x(16 * t + (lane >> 2), 16 * t + (lane < 16 ? lane : 0));
  }

  // Runs over a sequence of whole groups with three cursors on it, of one type:
  // one for the weights (two groups ahead), one for A (one ahead), one for the
  // products.  A cursor has bool more(), void next(), int64_t c() (the group's
  // first chunk), WPtr w(), XPtr x(int row, int scale_row), int rows();
  // done(cursor) is called after each group's products.  The cursors that run ahead stop at the last
  // group and load it again.
  template <class Cursor, class Done>
  static __device__ __forceinline__ void stream(f32x4 (&acc)[NS][MT], char* lds, Cursor cc, const WOff& wo,
                                                int64_t xpart, int64_t K, int lane, const Done& done) {
    if (!cc.more()) return;
    Cursor wc = cc, xc = cc;
    auto ahead = [](Cursor& c) {
      Cursor n = c;
      n.next();
      if (n.more()) c = n;
    };
    WRegs w0, w1;
    XAhead x[XT];
    auto load_ahead = [&] {
      if constexpr (FEW) {
        load_few<false>(x[0], xc, 0, xpart, K, lane);
      } else {
#pragma unroll
        for (int t = 0; t < XT; ++t) load_x(x[t], tile(xc, t, lane), xpart, xc.c(), lane);
      }
    };
    load_w(w0, wc.w(), wo, wc.c());
    ahead(wc);
    load_ahead();
    ahead(xc);
    load_w(w1, wc.w(), wo, wc.c());
    ahead(wc);
    auto step = [&](WRegs& w) {
      XFrags f[XT];
      stage_w(lds, w, lane);
      const bool is_wide = wide(w, lane);
      if constexpr (FEW) {
        store_few(lds, x[0], 0, lane);
        fetch_few<false>(lds, cc, 0, FR, xpart, K, lane);
        read_few(f[0], lds, lane);
      } else {
#pragma unroll
        for (int t = 0; t < XT; ++t) turn(f[t], lds, x[t], lane);
      }
      load_ahead();
      ahead(xc);
      load_w(w, wc.w(), wo, wc.c());
      ahead(wc);
      mma_all<0>(acc, lds, f, is_wide, lane);
      more_tiles<1, false>(acc, lds, cc, xpart, K, is_wide, lane);
      done(cc);
      cc.next();
    };
    while (true) {
      step(w0);
      if (!cc.more()) break;
      step(w1);
      if (!cc.more()) break;
    }
  }

  // The partial group at the cursor (its c() is the first chunk behind the whole
  // groups).
  template <class Cursor>
  static __device__ __forceinline__ void finish(f32x4 (&acc)[NS][MT], char* lds, const Cursor& cc, const WOff& wo,
                                                int64_t xpart, int64_t K, int lane) {
    WRegs w;
    XFrags f[XT];
    load_w_rest(w, cc.w(), wo, cc.c(), K, lane);
    stage_w(lds, w, lane);
    const bool is_wide = wide(w, lane);
    if constexpr (FEW) {
      fetch_few<true>(lds, cc, 0, 0, xpart, K, lane);
      read_few(f[0], lds, lane);
    } else {
#pragma unroll
      for (int t = 0; t < XT; ++t) {
        XRegs x;
        load_x_rest(x, tile(cc, t, lane), xpart, cc.c(), K, lane);
        turn(f[t], lds, x, lane);
      }
    }
    mma_all<0>(acc, lds, f, is_wide, lane);
    more_tiles<1, true>(acc, lds, cc, xpart, K, is_wide, lane);
  }

  // A cursor over every `stride`-th of `n` groups of one product.
  template <class Rows>
  struct Line {
    int64_t g, n, stride;
    const WPtr* wp;
    const Rows* addr;
    int n_rows;
    __device__ __forceinline__ bool more() const { return g < n; }
    __device__ __forceinline__ void next() { g += stride; }
    __device__ __forceinline__ int64_t c() const { return g * UC; }
    __device__ __forceinline__ const WPtr& w() const { return *wp; }
    __device__ __forceinline__ XPtr x(int row, int scale_row = 0) const { return (*addr)(row, scale_row); }
    __device__ __forceinline__ int rows() const { return n_rows; }
  };

  // Part `part` of `parts` of the sums over K, for n_rows rows of A whose
  // addresses addr(row, scale_row) gives.  The parts take the groups in turn, the partial one too.
  template <class Rows>
  static __device__ __forceinline__ void run(f32x4 (&acc)[NS][MT], char* lds, const WPtr& wp, const WOff& wo,
                                             const Rows& addr, int64_t xpart, int part, int parts, int64_t K,
                                             int n_rows, int lane) {
    const int64_t n = groups(K);
    stream(acc, lds, Line<Rows>{part, n, parts, &wp, &addr, n_rows}, wo, xpart, K, lane, [](const Line<Rows>&) {});
    if (rest(K) && part == (int)(n % parts))
      finish(acc, lds, Line<Rows>{n, n + 1, parts, &wp, &addr, n_rows}, wo, xpart, K, lane);
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
template <int XF, int DT, int NS, int MT, int UC, int NW, bool FEW = false>
__global__ __launch_bounds__(64 * NW) void mx4_strip_kernel(StripArgs a) {
  using S = Strip<SW_MX4, XF, NS, MT, UC, MT, FEW>;
  constexpr int TILES = NS * MT;
  __shared__ union {
    char wave[NW][S::LDS];
    f32x4 part[NW * TILES * 64];
  } sh;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NS), m0 = (int64_t)blockIdx.y * (16 * MT);
  const typename S::WPtr w{a.b + n0 * a.ldb, a.bs + n0 * a.ldbs};
  const typename S::WOff wo = S::offsets(a.N - n0, 16, a.ldb, a.ldbs, lane);
  const int64_t left = a.M - m0;
  auto rows = [&](int row, int scale_row) {
    const int64_t m = row < left ? row : left - 1, ms = scale_row < left ? scale_row : left - 1;
    typename S::XPtr x;
    x.x = a.a + m0 * a.lda;
    x.s = S::X4 ? a.as + m0 * a.ldas : nullptr;
    x.xo = (uint32_t)(m * a.lda);
    x.so = (uint32_t)(ms * a.ldas);
    return x;
  };
  f32x4 acc[NS][MT];
  S::clear(acc);
  S::run(acc, sh.wave[wave], w, wo, rows, 0, wave, NW, a.K,
         left >= 16 * MT ? 16 * MT : (int)left, lane);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) sh.part[(wave * TILES + i * MT + t) * 64 + lane] = acc[i][t];
  __syncthreads();
  for (int tile = wave; tile < TILES; tile += NW) {
    const f32x4 v = sum_waves(sh.part + tile * 64, TILES * 64, NW, lane);
    const int i = tile / MT, t = tile % MT;
    const int64_t m = m0 + 16 * t + (lane & 15), n = n0 + 16 * i + 4 * (lane >> 4);
    if (m < a.M && n < a.N) {
      uint16_t* c = a.c + m * a.ldc + n;
      uint16_t h[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) h[r] = cvt_out<DT>(v[r]);
      if (n + 4 <= a.N) {
        gstore(c, u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16});
      } else {
        for (int r = 0; r < 4 && n + r < a.N; ++r) gstore<uint16_t>(c + r, h[r]);
      }
    }
  }
}

}  // namespace gemmf16
