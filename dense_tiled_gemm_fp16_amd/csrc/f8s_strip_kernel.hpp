// FP8 products scaled by blocks with few rows of A (gfx950): f8s_tile_kernel.hpp's
// arithmetic, where the time goes to reading B once.
//
// A workgroup takes a strip of 16 NS columns and 16 MT rows; its waves share out
// the blocks of K in turn, each with a ring of D stages of LDS of its own, so the
// loop has no barriers and NW x D blocks of every strip are in flight.  The DMA
// brings whole lines (8 rows x 128 bytes an instruction) and does the turn into
// the matrix instruction's operand order, which loads into registers would pay
// for by touching 16 rows in every 16 lanes.  The waves' sums are added through
// LDS at the end, in ascending order.
//
// Bound by the latency of one pass of loads: 1 x 2048 x 7168 5.4 us in a graph
// (14.7 MB), 64 x 7168 x 2048 5.5, 512 x 2048 x 7168 18; a tile per workgroup without
// the split of K takes 31 us and more for 7168 k.
#pragma once

#include "f8s_big_kernel.hpp"

namespace gemmf16 {

template <int MT_, int NS_, int D_, int NW_>
struct F8sStrip {
  static constexpr int MT = MT_, NS = NS_, D = D_, NW = NW_, NT = 64 * NW;
  static constexpr int A_BYTES = MT * 2048, B_BYTES = NS * 2048, STAGE = A_BYTES + B_BYTES + 512;
  static constexpr int PER_STEP = 2 * MT + 2 * NS + 2;
  static constexpr int SUMS = NW * MT * NS * 1024;
  static constexpr int LDS = NW * D * STAGE > SUMS ? NW * D * STAGE : SUMS;
  static_assert(LDS <= 160 * 1024, "LDS budget");
};

template <class CF, int FA, int FB, bool ROWB, bool WIDE>
__global__ __launch_bounds__(CF::NT) void f8s_strip_kernel(F8sArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[CF::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * CF::NS), m0 = (int64_t)blockIdx.y * (16 * CF::MT);

  // This wave's blocks: wave, wave + NW, .. of the whole ones; ahead of them the
  // partial one, if its turn comes to this wave.
  const int64_t nf = a.K / 128;
  const int rem = (int)(a.K - nf * 128);
  const bool tail = rem > 0 && (int)(nf % CF::NW) == wave;
  const int64_t nq = (nf > wave ? (nf - wave + CF::NW - 1) / CF::NW : 0) + tail;
  auto block = [&](int64_t q) { return q < (int64_t)tail ? nf : wave + (q - tail) * CF::NW; };

  // Rows of this lane's DMA: 8 an instruction, lane l row l / 8, slot l % 8;
  // uniform bases, 32-bit offsets.  In the partial block chunks behind K read
  // the block's first one.
  constexpr int NI = 2 * (CF::MT + CF::NS);
  const char* const pa = uniform_ptr(a.A + m0 * a.lda - kSBias);
  const char* const pb = uniform_ptr(a.B + n0 * a.ldb - kSBias);
  auto chunk = [&](int i) { return (lane % 8) ^ f16r((i & 1) * 8 + lane / 8); };
  uint32_t off[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const bool is_a = i < 2 * CF::MT;
    const int64_t r = (is_a ? i : i - 2 * CF::MT) * 8 + lane / 8, left = (is_a ? a.M - m0 : a.N - n0) - 1;
    off[i] = (uint32_t)((r < left ? r : left) * (is_a ? a.lda : a.ldb) + (tail ? tail_chunk(chunk(i), rem) : 16 * chunk(i)) +
                        kSBias - 1024 * (i & 1));
  }
  const int64_t ma = m0 + lane < a.M ? m0 + lane : a.M - 1, nl = n0 + lane < a.N ? n0 + lane : a.N - 1;
  const char* const psa = uniform_ptr((const char*)(a.SA + m0 * a.sa_m));
  const char* const psb = uniform_ptr((const char*)(a.SB + (n0 >> a.shift) * a.sb_n));
  const uint32_t osa = (uint32_t)(4 * (ma - m0) * a.sa_m);
  const uint32_t osb = (uint32_t)(4 * ((nl >> a.shift) - (n0 >> a.shift)) * a.sb_n);
  const int64_t sa_step = 4 * a.sa_k, sb_step = 4 * a.sb_k;

  char* const mine = smem + wave * (CF::D * CF::STAGE);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(mine));
  auto issue = [&](int64_t b, int slot) {
    const uint32_t st = lds0 + slot * CF::STAGE;
#pragma unroll
    for (int i = 0; i < NI; i += 2) dma16s_batch<2>(&off[i], (i < 2 * CF::MT ? pa : pb) + b * 128, st + i * 1024);
    dma4s(osa, psa + b * sa_step, st + CF::A_BYTES + CF::B_BYTES);
    dma4s(osb, psb + b * sb_step, st + CF::A_BYTES + CF::B_BYTES + 256);
  };

  f32x4 acc[CF::NS][CF::MT];
#pragma unroll
  for (int i = 0; i < CF::NS; ++i)
#pragma unroll
    for (int j = 0; j < CF::MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int c0 = (g ^ f16r(lr)) * 16, c1 = c0 ^ 64;
  auto read = [&](const char* rows, int i) {
    const char* row = rows + (16 * i + lr) * 128;
    return join8(*reinterpret_cast<const u32x4*>(row + c0), *reinterpret_cast<const u32x4*>(row + c1));
  };
  auto compute = [&](auto tail_tag, int slot) {
    constexpr bool TAIL = decltype(tail_tag)::value;
    auto part = [&](const i32x8& v) { return TAIL ? mask_block(v, g, rem) : v; };
    const char* st = mine + slot * CF::STAGE;
    const char* sc = st + CF::A_BYTES + CF::B_BYTES;
    const float sb = ROWB ? kF8sUp : *reinterpret_cast<const float*>(sc + 256) * kF8sUp;
    F8sFrag<WIDE> fb[CF::NS];
#pragma unroll
    for (int i = 0; i < CF::NS; ++i) fb[i] = f8s_frag<WIDE, FB>(part(read(st + CF::A_BYTES, i)));
#pragma unroll
    for (int j = 0; j < CF::MT; ++j) {
      const F8sFrag<WIDE> fm = f8s_frag<WIDE, FA>(part(read(st, j)));
      const float s = *reinterpret_cast<const float*>(sc + (16 * j + lr) * 4) * sb;
      f32x4 d[CF::NS];
#pragma unroll
      for (int i = 0; i < CF::NS; ++i) d[i] = f8s_block<FA, FB>(fb[i], fm);
#pragma unroll
      for (int i = 0; i < CF::NS; ++i) {
        f32x4 sn{1.0f, 1.0f, 1.0f, 1.0f};
        if constexpr (ROWB) sn = *reinterpret_cast<const f32x4*>(sc + 256 + (16 * i + 4 * g) * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_fmaf(d[i][e], ROWB ? s * sn[e] : s, acc[i][j][e]);
      }
    }
  };

  if (nq > 0) issue(block(0), 0);
  if (tail) {
#pragma unroll
    for (int i = 0; i < NI; ++i) off[i] += 16 * chunk(i) - tail_chunk(chunk(i), rem);
  }
#pragma unroll
  for (int q = 1; q < CF::D; ++q)
    if (q < nq) issue(block(q), q);
  int slot = 0;
  auto step = [&](auto tail_tag, int64_t q) {
    // Blocks behind this one that are in flight: D - 1, fewer at the end.
    const int64_t left = nq - 1 - q;
    if (CF::D >= 4 && left >= 3)
      wait_vmcnt<3 * CF::PER_STEP>();
    else if (CF::D >= 3 && left >= 2)
      wait_vmcnt<2 * CF::PER_STEP>();
    else if (CF::D >= 2 && left >= 1)
      wait_vmcnt<CF::PER_STEP>();
    else
      wait_vmcnt<0>();
    compute(tail_tag, slot);
    wait_lgkmcnt0();               // read, so that the stage may be loaded again
    if (q + CF::D < nq) issue(block(q + CF::D), slot);
    slot = slot == CF::D - 1 ? 0 : slot + 1;
  };
  // The partial block ahead of the loop: within it the running sums would change registers.
  if (tail) step(std::true_type{}, 0);
  for (int64_t q = tail; q < nq; ++q) step(std::false_type{}, q);

  // The waves' sums: [wave][i][j][lane], then each 16 x 16 block's by one wave.
  __syncthreads();
  f32x4* const sums = reinterpret_cast<f32x4*>(smem);
#pragma unroll
  for (int i = 0; i < CF::NS; ++i)
#pragma unroll
    for (int j = 0; j < CF::MT; ++j) sums[(wave * (CF::NS * CF::MT) + i * CF::MT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int q = wave; q < CF::NS * CF::MT; q += CF::NW) {
    const int i = q / CF::MT, j = q % CF::MT;
    f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < CF::NW; ++w) v += sums[(w * (CF::NS * CF::MT) + q) * 64 + lane];
    const int64_t m = m0 + 16 * j + lr, n = n0 + 16 * i + 4 * g;
    int which = 0;                 // elements that did not stay finite
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] *= kF8sDown;
      if (m < a.M && n + e < a.N && !__builtin_isfinite(v[e])) which |= 1 << e;
    }
    if (__builtin_expect(__any(which != 0), 0)) {
      const F8sArgs b = f8s_args_again();
      const uint32_t rows = f8s_nan_rows(b, m0 + 16 * j, lane), cols = f8s_nan_cols(b, n0 + 16 * i, lane);
      which = rows >> lr & 1 ? 0 : which & (int)~(cols >> (4 * g));      // the others are NaN
      if (__any(which != 0)) {
        const f32x4 w = f8s_again<FA, FB, WIDE>(b, m0 + 16 * j, n0 + 16 * i, which, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = which >> e & 1 ? w[e] : v[e];
      }
    }
    if (m < a.M && n < a.N) store_out4(a.C, a.out, m * a.ldc + n, v, a.N - n);
  }
}

}  // namespace gemmf16
