// Product of two FP8 matrices with a float32 scale for each block of 128 along
// K (gfx950), by tiles:
// C[m,n] = sum over blocks b of sA[m,b] sB[n,b] sum over the block's k of a b.
//
// A step is one block, 128 k: the block's sum comes out of the matrix core on
// its own (v_mfma_f32_16x16x128_f8f6f4 from a zero accumulator, one instruction
// per 16 x 16 outputs) and four fused multiply-adds per lane bring it into the
// running sum at the product of its two scales.  Those take half the vector
// unit's cycles that the instruction takes of the matrix core's, so they fit
// beside it as long as the result is not awaited: a group of four instructions
// is issued before the first result is used.
//
//   LDS    S stages of 128 k: BM rows of A and BN rows of B, 128 bytes each, the
//          16-byte chunks of a row permuted against bank conflicts, and a dword
//          of scale for each row.  All comes by LDS-DMA (8 whole lines an
//          instruction; the scales as one dword a lane, so that any strides will
//          do).  Step t + S - 1 is issued into the stage of step t - 1 behind the
//          one barrier of step t.
//   k      a lane of group g = lane / 16 takes chunks g and g + 4 of its row,
//          for A and B alike: any assignment of k to bytes that both share is
//          the product.
//   sums   the first operand is B: a lane holds columns 4 (lane / 16) .. + 3 of
//          row lane % 16 of C, so one multiplication gives the scale of a row
//          and a block of columns, and 8 or 16 consecutive bytes are stored.
//   range  the product of two scales may leave float32's range where the block's sum,
//          which is 0 or between 2^-32 and 2^39, brings the result back into it.  So
//          the running sums are kept 2^40 times as large: what a product of scales
//          loses below 2^-126 is then, times such a sum, less than half a step of the
//          smallest float32.  The few sums that do not stay finite so, which lie above
//          2^88, meet scales above it or end as infinities or NaN, are formed again in
//          64 bits (f8s_again).  One multiplication a step and three for two outputs:
//          1 x 2048 x 7168 5.4 us instead of 5.3, 20864 x 1664 x 224 28.0 instead of
//          26.8, 32768 x 2048 x 7168 the same; with a NaN in every tile 8 to 16% more,
//          with all results above 2^88 twenty times as long.
//
// What bounds it: a step's data, which two stages give one step's time to arrive,
// and for float32 results the vector unit's instructions (256 beside 64 matrix
// instructions of 16 cycles).  Where the LDS holds two workgroups a compute unit
// takes two, whose barriers do not coincide: the 128 x 128 tile is four waves of
// 64 x 64 and two stages, 2048 x 7168 x 8192 in 138 us (1740 TFLOP/s; square
// blocks) and 165 (row blocks).  Eight waves of 32 x 64 with four stages took 206
// and 250, a 256 x 128 tile alone on its unit 167 and 187.
//
// A partial block at the end is a step like the others, its bytes behind K
// cleared in the registers on both sides; rows past M or N read the last valid
// row and are never stored.
//
// float32 results (WIDE): the FP8 matrix instructions add products in groups of
// 8, aligned to the group's largest and cut 2^-13 below it (measured; the older
// and the newer ones alike), which leaves sums of 1 to 3 in 10^5 of their
// size: far below a 16-bit result's last place, but not a float32 one's.  Those go
// through binary16, which holds every 8-bit value, at half the rate: 253 us
// (950 TFLOP/s; 200 on zeros, so the power it takes counts too).  Matrix
// instructions of 32 x 32 with their longer sums did not fit the registers.
#pragma once

#include "f8_kernel.hpp"
#include "mx4_common.hpp"

namespace gemmf16 {

enum F8sOut { F8S_F16 = 0, F8S_BF16 = 1, F8S_F32 = 2 };

struct F8sArgs {
  const char* A;
  int64_t lda;              // bytes
  const float* SA;
  int64_t sa_m, sa_k;       // elements, from row to row and from block to block
  const char* B;
  int64_t ldb;
  const float* SB;
  int64_t sb_n, sb_k;       // from scale row to scale row (n >> shift)
  void* C;
  int64_t ldc;              // elements
  int64_t M, N, K;
  int64_t GM, GN;
  int32_t panel, out, shift;
};

template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct F8sCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN, NT = 64 * NW, STAGES = STAGES_;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  // scale instructions: 64 rows each, as many per wave for every wave
  static constexpr int SI = ((BM + 63) / 64 + (BN + 63) / 64 + NW - 1) / NW;
  static constexpr int S_BYTES = SI * NW * 256;
  static constexpr int SB_AT = (BM + 63) / 64 * 256;         // B's scales behind A's
  static constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES, LDS = STAGES * STAGE;
  static constexpr int PER_CU = LDS <= 80 * 1024 ? 2 : 1, WAVES = PER_CU * NW / 4;   // workgroups a CU, waves a SIMD
  static constexpr int DMA_A = A_BYTES / 1024, DMA_B = B_BYTES / 1024;   // instructions of the workgroup
  static constexpr int DI = (DMA_A + DMA_B) / NW;                        // per wave
  static constexpr int BATCH = DI % 4 == 0 ? 4 : 2, BATCHES = DI / BATCH;
  static constexpr int PER_STEP = DI + SI;
  static_assert(DI % 2 == 0 && DMA_A % BATCH == 0, "batches of one operand");
  static_assert((DMA_A + DMA_B) % NW == 0 && TM % 16 == 0 && TN % 16 == 0 && 128 % TN == 0, "shape");
  static_assert(LDS <= 160 * 1024 && BM * BN * 4 <= LDS, "LDS budget, staging space");
};

// An operand's 32 bytes of a lane: as they are, or widened to binary16.
template <bool WIDE>
struct F8sFrag {
  i32x8 v;
};
template <>
struct F8sFrag<true> {
  f16x8 v[4];
};
// Two 8-bit elements of w (its low or high half) as binary16, exactly.
template <int F, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  if constexpr (F == F8_E4M3)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  else   // binary16's upper byte
    return __builtin_amdgcn_perm(w, 0u, HI ? 0x07000600u : 0x05000400u);
}
template <bool WIDE, int F>
__device__ __forceinline__ F8sFrag<WIDE> f8s_frag(const i32x8& b) {
  F8sFrag<WIDE> f;
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = (uint32_t)b[2 * i], hi = (uint32_t)b[2 * i + 1];
      f.v[i] = __builtin_bit_cast(f16x8, u32x4{widen2<F, false>(lo), widen2<F, true>(lo), widen2<F, false>(hi),
                                               widen2<F, true>(hi)});
    }
  } else {
    f.v = b;
  }
  return f;
}

// Sum over a block's 128 k, from zero; first operand the B block.
template <int FA, int FB>
__device__ __forceinline__ f32x4 f8s_block(const F8sFrag<true>& b, const F8sFrag<true>& a) {
  f32x4 d{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(b.v[i], a.v[i], d, 0, 0, 0);
  return d;
}
template <int FA, int FB>
__device__ __forceinline__ f32x4 mfma_f8_block(const i32x8& b, const i32x8& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, FB, FA, 0, 0, 0, 0);
}

template <int FA, int FB>
__device__ __forceinline__ f32x4 f8s_block(const F8sFrag<false>& b, const F8sFrag<false>& a) {
  return mfma_f8_block<FA, FB>(b.v, a.v);
}

// 4 consecutive outputs of a row, the first nv of them.
template <class T>
__device__ __forceinline__ void store4_part(T* p, const T (&v)[4], int nv) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < nv) gstore<T>(p + e, v[e]);
}
__device__ __forceinline__ void store_out4(void* C, int out, int64_t at, f32x4 v, int64_t nv) {
  if (out == F8S_F32) {
    float* p = (float*)C + at;
    if (nv >= 4) {
      gstore<f32x4>(p, v);
    } else {
      const float f[4] = {v[0], v[1], v[2], v[3]};
      store4_part(p, f, (int)nv);
    }
    return;
  }
  uint16_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = out == F8S_F16 ? cvt_out<DT_F16>(v[e]) : cvt_out<DT_BF16>(v[e]);
  uint16_t* p = (uint16_t*)C + at;
  if (nv >= 4)
    gstore<u32x2>(p, u32x2{(uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16)});
  else
    store4_part(p, h, (int)nv);
}

// A wave's block of TM rows x RB bytes, staged in LDS (16-byte chunk c of row r in
// place c ^ r % (RB / 16)), to C by whole rows.  Stored from the sums, 8 or 16 bytes
// into each of 16 rows, a tile's end costs a request per piece: 16384 x 4096 x 128
// took 48 us so and takes 35, 11008 x 4730 x 258 52 and 46 (128 x 128 tiles).  The first
// `rows` rows and `bytes` bytes of each lie inside C (none, if negative); any alignment.
template <int TM, int RB>
__device__ __forceinline__ void store_staged_block(char* C, int64_t pitch, int64_t rows, int64_t bytes, const char* stage,
                                                   int lane) {
  constexpr int CH = RB / 16, PER = 64 / CH;
  const int c = lane % CH, r0 = lane / CH;
  auto chunk = [&](int r) { return *reinterpret_cast<const u32x4*>(stage + r * RB + ((c ^ (r & (CH - 1))) << 4)); };
  C += r0 * pitch + 16 * c;
  if (rows >= TM && bytes >= RB) {
#pragma unroll
    for (int it = 0; it < TM / PER; ++it) gstore<u32x4>(C + it * PER * pitch, chunk(PER * it + r0));
    return;
  }
  const int n = (int)(bytes < RB ? bytes : RB) - 16 * c, last = (int)(rows < TM ? rows : TM) - r0;
#pragma unroll
  for (int it = 0; it < TM / PER; ++it) {
    const u32x4 v = chunk(PER * it + r0);
    char* const p = C + it * PER * pitch;
    if (PER * it < last) {
      if (n >= 16) {
        gstore<u32x4>(p, v);
      } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
          if (2 * e < n) gstore<uint16_t>((uint16_t*)p + e, (uint16_t)(v[e / 2] >> (16 * (e % 2))));
      }
    }
  }
}

// Bytes of a lane's 32 that lie behind rem, zeroed (those at k >= rem of the block:
// chunk g is k 16 g .., chunk g + 4 k 64 + 16 g ..).
__device__ __forceinline__ i32x8 mask_block(i32x8 v, int g, int rem) {
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const int n = rem - (16 * g + 4 * (w & 3) + (w < 4 ? 0 : 64));
    v[w] = n >= 4 ? v[w] : (n <= 0 ? 0 : (v[w] & ((1 << (8 * n)) - 1)));
  }
  return v;
}

// The running sums are this much larger than the results (the comment at the top).
constexpr float kF8sUp = 0x1p40f, kF8sDown = 0x1p-40f;

// Sums to results.  Returns, to the whole wave, whether any of its elements did not stay
// finite; bit i FM + j of odd[e] tells that element e of sums[i][j] did not.  (Products of
// two results add up to a finite number only if all are; where they do not, each result
// is looked at.)
template <int FN, int FM>
__device__ __forceinline__ bool f8s_bring_down(f32x4 (&sums)[FN][FM], uint32_t (&odd)[4]) {
  static_assert(FN * FM <= 32, "bits of a flag");
  float z[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sums[i][j][e] *= kF8sDown;
#pragma unroll
      for (int h = 0; h < 2; ++h) z[h] = __builtin_fmaf(sums[i][j][2 * h], sums[i][j][2 * h + 1], z[h]);
    }
  odd[0] = odd[1] = odd[2] = odd[3] = 0;
  if (__builtin_expect(!__any(!__builtin_isfinite(z[0]) || !__builtin_isfinite(z[1])), 1)) return false;
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!__builtin_isfinite(sums[i][j][e])) odd[e] |= 1u << (i * FM + j);
  return __any((odd[0] | odd[1] | odd[2] | odd[3]) != 0);
}

// Of 16 rows (or columns), which have a NaN scale, a bit each: lane l looks at every
// fourth scale, from l / 16 on, of row l % 16, which begin at s.
__device__ __forceinline__ uint32_t f8s_nan_scales(const float* s, int64_t step, int64_t blocks, int lane) {
  bool bad = false;
#pragma unroll 4
  for (int64_t b = lane >> 4; b < blocks; b += 4) {
    const float v = s[b * step];
    bad |= v != v;
  }
  const uint64_t m = __ballot(bad);
  return (uint32_t)(m | m >> 16 | m >> 32 | m >> 48) & 0xFFFFu;
}
__device__ __forceinline__ int64_t f8s_below(int64_t i, int64_t n) { return i < n ? i : n - 1; }
__device__ __forceinline__ uint32_t f8s_nan_rows(const F8sArgs& a, int64_t m0, int lane) {
  return f8s_nan_scales(a.SA + f8s_below(m0 + (lane & 15), a.M) * a.sa_m, a.sa_k, (a.K + 127) / 128, lane);
}
__device__ __forceinline__ uint32_t f8s_nan_cols(const F8sArgs& a, int64_t n0, int lane) {
  return f8s_nan_scales(a.SB + (f8s_below(n0 + (lane & 15), a.N) >> a.shift) * a.sb_n, a.sb_k, (a.K + 127) / 128, lane);
}

// A block of 16 rows from m0 (inside A) x 16 columns from n0 (inside C) again, its sums
// in 64 bits; only the elements with a bit in `which` count (column n0 + 4 (lane / 16) +
// e of row m0 + lane % 16).  Straight from memory, a step at a time: 1 us a step.
template <int FA, int FB, bool WIDE>
__device__ __forceinline__ f32x4 f8s_again(const F8sArgs& a, int64_t m0, int64_t n0, int which, int lane) {
  const int lr = lane & 15, g = lane >> 4;
  const int64_t m = f8s_below(m0 + lr, a.M), n = f8s_below(n0 + lr, a.N);
  const char* pa = a.A + m * a.lda + 16 * g;
  const char* pb = a.B + n * a.ldb + 16 * g;
  const float* sa = a.SA + m * a.sa_m;
  const float* sb[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sb[e] = a.SB + (f8s_below(n0 + 4 * g + e, a.N) >> a.shift) * a.sb_n;
  double v[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 1
  for (int64_t k = 0; k < a.K; k += 128) {
    const int rem = a.K - k < 128 ? (int)(a.K - k) : 128;
    auto part = [&](const char* p) {
      return mask_block(join8(16 * g < rem ? load16(p) : zero4(), 64 + 16 * g < rem ? load16(p + 64) : zero4()), g, rem);
    };
    const f32x4 d = f8s_block<FA, FB>(f8s_frag<WIDE, FB>(part(pb)), f8s_frag<WIDE, FA>(part(pa)));
    const double s = *sa;
    int left = 0;                                           // NaN stays NaN
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __builtin_fma((double)d[e] * s, (double)*sb[e], v[e]);
      left |= v[e] == v[e] ? 1 << e : 0;
      sb[e] += a.sb_k;
    }
    if (!__any((left & which) != 0)) break;
    pa += 128;
    pb += 128;
    sa += a.sa_k;
  }
  return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

// The kernel's arguments, loaded again where few calls come: what would be kept of
// them costs the others scalar registers.
__device__ __forceinline__ F8sArgs f8s_args_again() {
  const char __attribute__((address_space(4)))* p =
      (const char __attribute__((address_space(4)))*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  F8sArgs a;
  __builtin_memcpy(&a, (const void*)p, sizeof(a));
  return a;
}

// The elements of a wave's FN x FM blocks from row m0 and column n0 that did not stay
// finite, over what was stored in their place; but for those of rows and columns with a
// NaN scale, which are NaN.
template <int FA, int FB, bool WIDE, int FN, int FM>
__device__ __forceinline__ void f8s_store_again(int64_t m0, int64_t n0, const uint32_t (&odd)[4], int lane) {
  static_assert(FM <= 4, "rows in 64 bits");
  const F8sArgs a = f8s_args_again();
  wait_vmcnt<0>();
  uint64_t rows = 0;
#pragma unroll 1
  for (int j = 0; j < FM; ++j) rows |= (uint64_t)f8s_nan_rows(a, m0 + 16 * j, lane) << (16 * j);
#pragma unroll 1
  for (int i = 0; i < FN; ++i) {
    const int64_t n = n0 + 16 * i + 4 * (lane >> 4);
    const uint32_t cols = f8s_nan_cols(a, n0 + 16 * i, lane) >> (4 * (lane >> 4));
#pragma unroll 1
    for (int j = 0; j < FM; ++j) {
      const int64_t m = m0 + 16 * j + (lane & 15);
      int which = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) which |= n + e < a.N ? (int)(odd[e] >> (i * FM + j) & 1u) << e : 0;
      which = m < a.M && !(rows >> (16 * j + (lane & 15)) & 1) ? which & (int)~cols : 0;
      if (!__any(which != 0)) continue;
      const f32x4 v = f8s_again<FA, FB, WIDE>(a, m0 + 16 * j, n0 + 16 * i, which, lane);
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const float f = e == 0 ? v[0] : e == 1 ? v[1] : e == 2 ? v[2] : v[3];
        if (which >> e & 1) store_out4(a.C, a.out, m * a.ldc + n + e, f32x4{f, f, f, f}, 1);
      }
    }
  }
}

// Offset of a DMA lane's chunk c in a block of which rem bytes are left: chunks
// wholly behind K read the block's first one (mask_block clears them; a chunk
// that K ends in is read whole, 16 aligned bytes of which one at least is K's).
__device__ __forceinline__ int tail_chunk(int c, int rem) { return 16 * c < rem ? 16 * c : 0; }

// 16-byte chunk c of row r lies in slot c ^ f16r(r): the same for every block of
// 16 rows, 16 rows reading one chunk fall on distinct banks.
__device__ __forceinline__ int f16r(int r) { return (r ^ (r >> 3 & 1)) & 7; }

// A wave's LDS-DMA of a step: DI instructions of 8 rows, A's first, in batches of
// one operand, then SI of 64 scales, A's first (the last may be one too many: it
// repeats B's rows).  Uniform bases, and 32-bit offsets of the lanes.
template <class CF>
struct F8sFeed {
  const char* src[CF::BATCHES];
  uint32_t off[CF::DI];
  const char* ssrc[CF::SI];
  uint32_t soff[CF::SI];
  int64_t sstep[CF::SI];
  int wave, lane, nf, rem, nb, at;      // whole blocks, k behind them, blocks, blocks issued
  uint32_t lds0;

  __device__ __forceinline__ int chunk(int i) const { return (lane % 8) ^ f16r((wave * CF::DI + i) * 8 + lane / 8); }

  __device__ __forceinline__ F8sFeed(const F8sArgs& a, int64_t m0, int64_t n0, const char* smem, int wave_, int lane_)
      : wave(wave_), lane(lane_), nf((int)(a.K / 128)), rem((int)(a.K % 128)), nb(nf + (rem > 0)), at(0),
        lds0(__builtin_amdgcn_readfirstlane(lds_addr(smem))) {
#pragma unroll
    for (int i = 0; i < CF::DI; ++i) {
      const int q = wave * CF::DI + i;
      const bool is_a = q < CF::DMA_A;
      const int64_t r = (is_a ? q : q - CF::DMA_A) * 8 + lane / 8, left = (is_a ? a.M - m0 : a.N - n0) - 1;
      if (i % CF::BATCH == 0) src[i / CF::BATCH] = uniform_ptr((is_a ? a.A + m0 * a.lda : a.B + n0 * a.ldb) - kSBias);
      off[i] = (uint32_t)((r < left ? r : left) * (is_a ? a.lda : a.ldb) +
                          (nf > 0 ? 16 * chunk(i) : tail_chunk(chunk(i), rem)) + kSBias - 1024 * (i % CF::BATCH));
    }
#pragma unroll
    for (int i = 0; i < CF::SI; ++i) {
      const int q = wave * CF::SI + i;
      const bool is_a = q < (CF::BM + 63) / 64;
      const int64_t last = (is_a ? a.M : a.N) - 1, row = is_a ? m0 + q * 64 : n0 + (q - (CF::BM + 63) / 64) * 64;
      const int64_t r0 = row < last ? row : last, r1 = row + lane < last ? row + lane : last;
      ssrc[i] = uniform_ptr((const char*)(is_a ? a.SA + r0 * a.sa_m : a.SB + (r0 >> a.shift) * a.sb_n));
      soff[i] = (uint32_t)(4 * (is_a ? (r1 - r0) * a.sa_m : ((r1 >> a.shift) - (r0 >> a.shift)) * a.sb_n));
      sstep[i] = 4 * (is_a ? a.sa_k : a.sb_k);
    }
  }

  // The next step into `slot`, from bases that advance with each call but the last
  // block's (which is loaded again past the end, so that every step issues the
  // same number); ahead of a partial block the lanes' chunks are set for it.
  __device__ __forceinline__ void issue(int slot) {
    const uint32_t st = lds0 + slot * CF::STAGE;
#pragma unroll
    for (int i = 0; i < CF::BATCHES; ++i)
      dma16s_batch<CF::BATCH>(&off[i * CF::BATCH], src[i], st + (wave * CF::DI + i * CF::BATCH) * 1024);
#pragma unroll
    for (int i = 0; i < CF::SI; ++i)
      dma4s(soff[i], ssrc[i], st + CF::A_BYTES + CF::B_BYTES + (wave * CF::SI + i) * 256);
    if (++at < nb) {
#pragma unroll
      for (int i = 0; i < CF::BATCHES; ++i) src[i] += 128;
#pragma unroll
      for (int i = 0; i < CF::SI; ++i) ssrc[i] += sstep[i];
      if (rem > 0 && at == nf) {
#pragma unroll
        for (int i = 0; i < CF::DI; ++i) off[i] += tail_chunk(chunk(i), rem) - 16 * chunk(i);
      }
    }
  }
};

template <class CF, int FA, int FB, bool ROWB, bool WIDE>
__global__ __launch_bounds__(CF::NT, CF::WAVES) void f8s_tile_kernel(F8sArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[CF::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / CF::WN, wn = wave % CF::WN;
  const int lr = lane & 15, g = lane >> 4;

  int64_t pm, pn;
  raster_tile(blockIdx.x, a.GM, a.GN, a.panel, pm, pn);
  const int64_t m0 = pm * CF::BM, n0 = pn * CF::BN;
  F8sFeed<CF> feed(a, m0, n0, smem, wave, lane);
  const int nf = feed.nf, rem = feed.rem;

  // LDS addresses of stage 0: chunks g and g + 4 of row lr of a block of rows.
  const int c0 = (g ^ f16r(lr)) * 16, c1 = c0 ^ 64;
  const char* const la = smem + (wm * CF::TM + lr) * 128;
  const char* const lb = smem + CF::A_BYTES + (wn * CF::TN + lr) * 128;
  const char* const lsa = smem + CF::A_BYTES + CF::B_BYTES + (wm * CF::TM + lr) * 4;
  const char* const lsb = smem + CF::A_BYTES + CF::B_BYTES + CF::SB_AT + wn * CF::TN * 4;
  auto read = [&](const char* rows, int i) {
    const char* p = rows + i * 2048;
    return join8(*reinterpret_cast<const u32x4*>(p + c0), *reinterpret_cast<const u32x4*>(p + c1));
  };

  f32x4 acc[CF::FN][CF::FM];
#pragma unroll
  for (int i = 0; i < CF::FN; ++i)
#pragma unroll
    for (int j = 0; j < CF::FM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // One block of K: unit u multiplies block i = u / FM of B by block j = u % FM of
  // A, then the sums of the unit LAG before are taken to their scales.  A block
  // of B is read while the one before it is multiplied.
  constexpr int UNITS = CF::FN * CF::FM, LAG = UNITS > 3 ? 3 : UNITS - 1;
  auto compute = [&](auto tail_tag, int slot) {
    constexpr bool TAIL = decltype(tail_tag)::value;
    const char* const ra = la + slot * CF::STAGE;
    const char* const rb = lb + slot * CF::STAGE;
    const char* const rsa = lsa + slot * CF::STAGE;
    const char* const rsb = lsb + slot * CF::STAGE;
    auto part = [&](const i32x8& v) { return TAIL ? mask_block(v, g, rem) : v; };
    i32x8 next = part(read(rb, 0));
    F8sFrag<WIDE> fm[CF::FM], fb;
    float s[CF::FM];
    const float sb = ROWB ? kF8sUp : *reinterpret_cast<const float*>(rsb) * kF8sUp;
#pragma unroll
    for (int j = 0; j < CF::FM; ++j) {
      fm[j] = f8s_frag<WIDE, FA>(part(read(ra, j)));
      s[j] = *reinterpret_cast<const float*>(rsa + j * 64) * sb;
    }
    if constexpr (WIDE) {
      // Four instructions to a sum: those of a block of B's units in turn, so that
      // none waits for the one before it.
      f32x4 d[2][CF::FM], sn[2];
      auto add = [&](int i) {
#pragma unroll
        for (int j = 0; j < CF::FM; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] = __builtin_fmaf(d[i & 1][j][e], ROWB ? s[j] * sn[i & 1][e] : s[j], acc[i][j][e]);
      };
      fb = f8s_frag<WIDE, FB>(next);
#pragma unroll
      for (int i = 0; i < CF::FN; ++i) {
        if (i + 1 < CF::FN) next = part(read(rb, i + 1));
        if constexpr (ROWB) sn[i & 1] = *reinterpret_cast<const f32x4*>(rsb + i * 64 + 16 * g);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int j = 0; j < CF::FM; ++j)
            d[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                fb.v[q], fm[j].v[q], q == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : d[i & 1][j], 0, 0, 0);
        if (i > 0) add(i - 1);
        if (i + 1 < CF::FN) fb = f8s_frag<WIDE, FB>(next);
        __builtin_amdgcn_sched_barrier(0);
      }
      add(CF::FN - 1);
      return;
    }
    f32x4 d[LAG + 1], sn[2];
    if constexpr (ROWB) sn[0] = *reinterpret_cast<const f32x4*>(rsb + 16 * g);
#pragma unroll
    for (int u = 0; u < UNITS + LAG; ++u) {
      if (u < UNITS) {
        const int i = u / CF::FM, j = u % CF::FM;
        if (j == 0) {
          fb = f8s_frag<WIDE, FB>(next);
          if (i + 1 < CF::FN) next = part(read(rb, i + 1));
        }
        d[u % (LAG + 1)] = f8s_block<FA, FB>(fb, fm[j]);
      }
      if (u >= LAG) {
        const int v = u - LAG, i = v / CF::FM, j = v % CF::FM;
        if constexpr (ROWB)
          if (j == 0 && i + 1 < CF::FN) sn[(i + 1) & 1] = *reinterpret_cast<const f32x4*>(rsb + (i + 1) * 64 + 16 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_fmaf(d[v % (LAG + 1)][e], ROWB ? s[j] * sn[i & 1][e] : s[j], acc[i][j][e]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

#pragma unroll
  for (int t = 0; t < CF::STAGES - 1; ++t) feed.issue(t);
  int slot = 0;
  for (int t = 0; t < nf; ++t) {
    wait_vmcnt<(CF::STAGES - 2) * CF::PER_STEP>();    // this wave's part of step t landed,
    wait_lgkmcnt0();                                  // and its reads of step t - 1 returned
    wg_barrier();                                     // both of every wave's
    feed.issue(slot == 0 ? CF::STAGES - 1 : slot - 1);
    __builtin_amdgcn_sched_barrier(0);
    compute(std::false_type{}, slot);
    slot = slot == CF::STAGES - 1 ? 0 : slot + 1;
  }
  if (rem > 0) {     // behind the loop: within it the running sums would change registers
    wait_vmcnt<(CF::STAGES - 2) * CF::PER_STEP>();
    wait_lgkmcnt0();
    wg_barrier();
    compute(std::true_type{}, slot);
  }
  wait_vmcnt<0>();       // no LDS transfer may outlive the workgroup, and every
  wait_lgkmcnt0();       // wave has read its stage: the LDS is free
  wg_barrier();
  uint32_t odd[4];
  const bool again = f8s_bring_down(acc, odd);
  char* const stage = smem + wave * (CF::TM * CF::TN * 4);
  const int64_t mw = m0 + wm * CF::TM, nw = n0 + wn * CF::TN, es = a.out == F8S_F32 ? 4 : 2;
  char* const cw = (char*)a.C + (mw * a.ldc + nw) * es;
  if (a.out == F8S_F32) {
#pragma unroll
    for (int j = 0; j < CF::FM; ++j)
#pragma unroll
      for (int i = 0; i < CF::FN; ++i) {
        const int r = j * 16 + lr, c = 4 * i + g;
        *reinterpret_cast<f32x4*>(stage + r * (CF::TN * 4) + ((c ^ (r & (CF::TN / 4 - 1))) << 4)) = acc[i][j];
      }
    store_staged_block<CF::TM, CF::TN * 4>(cw, a.ldc * 4, a.M - mw, (a.N - nw) * 4, stage, lane);
  } else {
    auto put = [&](auto dt_tag) {
      constexpr int DT = decltype(dt_tag)::value;
#pragma unroll
      for (int j = 0; j < CF::FM; ++j)
#pragma unroll
        for (int i = 0; i < CF::FN; ++i) {
          const int r = j * 16 + lr, c = 2 * i + (g >> 1);
          *reinterpret_cast<u32x2*>(stage + r * (CF::TN * 2) + ((c ^ (r & (CF::TN / 8 - 1))) << 4) + 8 * (g & 1)) =
              u32x2{pack_out2<DT>(acc[i][j][0], acc[i][j][1]), pack_out2<DT>(acc[i][j][2], acc[i][j][3])};
        }
    };
    if (a.out == F8S_F16)
      put(std::integral_constant<int, DT_F16>{});
    else
      put(std::integral_constant<int, DT_BF16>{});
    store_staged_block<CF::TM, CF::TN * 2>(cw, a.ldc * 2, a.M - mw, (a.N - nw) * 2, stage, lane);
  }
  if (again) f8s_store_again<FA, FB, WIDE, CF::FN, CF::FM>(mw, nw, odd, lane);
}

}  // namespace gemmf16
