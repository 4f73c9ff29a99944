// The 256 x 256 tile of the FP8 products scaled by blocks (gfx950): square
// blocks of B, 16-bit results (f8s_tile_kernel.hpp has the method).
//
// 8 waves of 64 x 128: 4 blocks of 16 rows of A (j) and 8 of B (i), 32 matrix
// instructions and 128 multiply-adds a step of 128 k.  The two stages that fit
// the LDS beside each other leave a step's time for a stage's transfer, so what
// counts is that every instruction of a step is issued where its operands have
// long been there.  The step is written out in that order:
//
//   units 0 .. 15    i = 0 .. 3, all j each: as a block of B is done with, the
//                    block four further on is read into its registers
//   units 16 .. 31   j = 0 .. 3, i = 5, 6, 7, 4 each: as a block of A is done
//                    with, the next step's is read into its registers, at the
//                    end the next step's first blocks of B too
//   each unit        one matrix instruction, then the multiply-adds of the unit
//                    three before, whose sum has arrived
//   after unit 18    all of this stage has been read, by every wave behind the
//                    barrier, and all of the next one has landed: the stage
//                    after that is loaded into this one
//
// Registers: 128 running sums, 4 sums of blocks in flight (16), A 32, B 5 blocks
// (40).  The stages' halves lie so that all LDS addresses of both are one base
// and an immediate; the loop takes two steps a turn.
//
// 32768 x 2048 x 7168 in 424 us (2270 TFLOP/s), 348 on zeros: the clock falls to
// 1.8 GHz at the power of multiplying random bytes, with the matrix core busy 55%
// of the cycles (the unscaled FP8 tile, without the multiply-adds: 373).  Touching
// the lines of later steps ahead of their transfer made it slower (432).
#pragma once

#include "f8s_tile_kernel.hpp"

namespace gemmf16 {

struct F8sBig {
  static constexpr int BM = 256, BN = 256, WAVES_M = 4, WAVES_N = 2, NW = 8, NT = 512;
  static constexpr int WTM = 64, WTN = 128, FM = 4, FN = 8;
  static constexpr int HALF = 256 * 128;                     // an operand's stage
  static constexpr int A_AT = 0, B_AT = 2 * HALF, S_AT = 4 * HALF, S_BYTES = 2048;
  static constexpr int LDS = S_AT + 2 * S_BYTES;
  static constexpr int PER_STEP = 9;                         // DMA instructions of a wave
  static_assert(LDS <= 160 * 1024, "LDS budget");
};

template <int FA, int FB, int DT>
__global__ __launch_bounds__(F8sBig::NT) void f8s_big_kernel(F8sArgs a) {
  using CF = F8sBig;
  __shared__ __attribute__((aligned(1024))) char smem[CF::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / CF::WAVES_N, wn = wave % CF::WAVES_N;
  const int lr = lane & 15, g = lane >> 4;

  int64_t pm, pn;
  raster_tile(blockIdx.x, a.GM, a.GN, a.panel, pm, pn);
  const int64_t m0 = pm * CF::BM, n0 = pn * CF::BN;

  // DMA: this wave's rows 32 w .. 32 w + 31 of both operands, 8 an instruction;
  // scales of rows 64 w .. of A (waves 0 .. 3) or B.  Offsets of 32 bits beside
  // uniform bases.
  const char* pa = uniform_ptr(a.A + m0 * a.lda - kSBias);
  const char* pb = uniform_ptr(a.B + n0 * a.ldb - kSBias);
  uint32_t oa[4], ob[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 32 * wave + 8 * i + lane / 8, c = (lane % 8) ^ f16r(r);
    const int64_t ma = m0 + r < a.M ? r : a.M - 1 - m0, nb = n0 + r < a.N ? r : a.N - 1 - n0;
    oa[i] = (uint32_t)(ma * a.lda + 16 * c + kSBias - 1024 * i);
    ob[i] = (uint32_t)(nb * a.ldb + 16 * c + kSBias - 1024 * i);
  }
  const bool sw_a = wave < 4;
  const int64_t srow = (sw_a ? m0 : n0) + 64 * (wave & 3);
  const int64_t slast = (sw_a ? a.M : a.N) - 1;
  const int64_t s0 = srow < slast ? srow : slast;             // the wave's first valid row
  const int64_t s1 = srow + lane < slast ? srow + lane : slast;
  const char* ps = uniform_ptr((const char*)(sw_a ? a.SA + s0 * a.sa_m : a.SB + (s0 >> a.shift) * a.sb_n));
  const uint32_t os = (uint32_t)(4 * (sw_a ? (s1 - s0) * a.sa_m : ((s1 >> a.shift) - (s0 >> a.shift)) * a.sb_n));
  const int64_t s_step = 4 * (sw_a ? a.sa_k : a.sb_k);

  const int nf = (int)(a.K / 128), rem = (int)(a.K - (int64_t)nf * 128);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  const uint32_t l_rows = lds0 + wave * 4096, l_scales = lds0 + CF::S_AT + wave * 256;

  f32x4 acc[CF::FN][CF::FM], d[4];
#pragma unroll
  for (int i = 0; i < CF::FN; ++i)
#pragma unroll
    for (int j = 0; j < CF::FM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // LDS addresses of stage 0: chunks g and g + 4 of row lr of a block.
  const char* const la = smem + CF::A_AT + (wm * CF::WTM + lr) * 128;
  const char* const lb = smem + CF::B_AT + (wn * CF::WTN + lr) * 128;
  const int c0 = (g ^ f16r(lr)) * 16, c1 = c0 ^ 64;
  const char* const a0 = la + c0;
  const char* const a1 = la + c1;
  const char* const b0 = lb + c0;
  const char* const b1 = lb + c1;
  const char* const sa = smem + CF::S_AT + (wm * CF::WTM + lr) * 4;
  const char* const sb = smem + CF::S_AT + 1024 + wn * CF::WTN * 4;
  auto read_a = [&](int slot, int j) {
    const int o = slot * CF::HALF + j * 2048;
    return join8(*reinterpret_cast<const u32x4*>(a0 + o), *reinterpret_cast<const u32x4*>(a1 + o));
  };
  auto read_b = [&](int slot, int i) {
    const int o = slot * CF::HALF + i * 2048;
    return join8(*reinterpret_cast<const u32x4*>(b0 + o), *reinterpret_cast<const u32x4*>(b1 + o));
  };

  i32x8 fm[4], x, y0, y1, y2, y3;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sn[4], sbn = 0.0f, s3 = 0.0f;   // s3: row block 3 of the step before

  // Unit u multiplies block IB[u] of B by block JA[u] of A.
  auto block_of = [](int u) constexpr { return u < 16 ? u / 4 : (u % 4 == 3 ? 4 : 5 + u % 4); };
  auto row_of = [](int u) constexpr { return u < 16 ? u % 4 : (u - 16) / 4; };

  auto step = [&](auto slot_tag, const char* na, const char* nb, const char* ns) {
    constexpr int S = decltype(slot_tag)::value, T = S ^ 1;
    auto unit = [&](auto u_tag, const i32x8& fb) {
      constexpr int u = decltype(u_tag)::value;
      constexpr int v = (u + 29) % 32;                        // three before
      constexpr int vi = block_of(v), vj = row_of(v);
      d[u % 4] = mfma_f8_block<FA, FB>(fb, fm[row_of(u)]);
      const float sv = u < 3 ? s3 : s[vj];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[vi][vj][e] = __builtin_fmaf(d[v % 4][e], sv, acc[vi][vj][e]);
      __builtin_amdgcn_sched_barrier(0);
    };
#define UNIT(U, F) unit(std::integral_constant<int, U>{}, F)
    UNIT(0, x);
    y3 = read_b(S, 4);
    UNIT(1, x);
    UNIT(2, x);
    UNIT(3, x);
    x = read_b(S, 5);
    UNIT(4, y0);
    UNIT(5, y0);
    UNIT(6, y0);
    UNIT(7, y0);
    y0 = read_b(S, 6);
    UNIT(8, y1);
    UNIT(9, y1);
    UNIT(10, y1);
    UNIT(11, y1);
    y1 = read_b(S, 7);
    UNIT(12, y2);
    UNIT(13, y2);
    UNIT(14, y2);
    UNIT(15, y2);
    UNIT(16, x);
    UNIT(17, y0);
    UNIT(18, y1);
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    wg_barrier();
    __builtin_amdgcn_sched_barrier(0);
    UNIT(19, y3);
    fm[0] = read_a(T, 0);
    dma16s_batch<4>(oa, na, l_rows + CF::A_AT + S * CF::HALF);
    UNIT(20, x);
    sbn = *reinterpret_cast<const float*>(sb + T * CF::S_BYTES);
#pragma unroll
    for (int j = 0; j < 4; ++j) sn[j] = *reinterpret_cast<const float*>(sa + T * CF::S_BYTES + j * 64);
    UNIT(21, y0);
    dma16s_batch<4>(ob, nb, l_rows + CF::B_AT + S * CF::HALF);
    UNIT(22, y1);
    y2 = read_b(T, 3);
    UNIT(23, y3);
    fm[1] = read_a(T, 1);
    UNIT(24, x);
    dma4s(os, ns, l_scales + S * CF::S_BYTES);
    UNIT(25, y0);
    UNIT(26, y1);
    UNIT(27, y3);
    fm[2] = read_a(T, 2);
    UNIT(28, x);
    x = read_b(T, 0);
    UNIT(29, y0);
    y0 = read_b(T, 1);
    UNIT(30, y1);
    y1 = read_b(T, 2);
    UNIT(31, y3);
    fm[3] = read_a(T, 3);
#undef UNIT
    s3 = s[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = sn[j] * (sbn * kF8sUp);
  };

  if (nf > 0) {
    const int64_t one = nf > 1 ? 1 : 0;
    dma16s_batch<4>(oa, pa, l_rows + CF::A_AT);
    dma16s_batch<4>(ob, pb, l_rows + CF::B_AT);
    dma4s(os, ps, l_scales);
    dma16s_batch<4>(oa, pa + one * 128, l_rows + CF::A_AT + CF::HALF);
    dma16s_batch<4>(ob, pb + one * 128, l_rows + CF::B_AT + CF::HALF);
    dma4s(os, ps + one * s_step, l_scales + CF::S_BYTES);
    wait_vmcnt<CF::PER_STEP>();
    wg_barrier();
#pragma unroll
    for (int j = 0; j < 4; ++j) fm[j] = read_a(0, j);
    x = read_b(0, 0);
    y0 = read_b(0, 1);
    y1 = read_b(0, 2);
    y2 = read_b(0, 3);
    sbn = *reinterpret_cast<const float*>(sb);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = *reinterpret_cast<const float*>(sa + j * 64) * (sbn * kF8sUp);
    // Sources of step t + 2; past the end the last step is loaded again, into a
    // stage that no step reads.
    const char* na = pa + (int64_t)(nf > 2 ? 2 : nf - 1) * 128;
    const char* nb = pb + (int64_t)(nf > 2 ? 2 : nf - 1) * 128;
    const char* ns = ps + (int64_t)(nf > 2 ? 2 : nf - 1) * s_step;
    auto next = [&](int t) {
      if (t + 3 < nf) {
        na += 128;
        nb += 128;
        ns += s_step;
      }
    };
    int t = 0;
    for (; t + 1 < nf; t += 2) {
      step(std::integral_constant<int, 0>{}, na, nb, ns);
      next(t);
      step(std::integral_constant<int, 1>{}, na, nb, ns);
      next(t + 1);
    }
    if (t < nf) step(std::integral_constant<int, 0>{}, na, nb, ns);
    // The last three units' sums (row block 3).
#pragma unroll
    for (int v = 29; v < 32; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[v == 31 ? 4 : 5 + v % 4][3][e] = __builtin_fmaf(d[v % 4][e], s3, acc[v == 31 ? 4 : 5 + v % 4][3][e]);
    wait_vmcnt<0>();
  }
  wait_lgkmcnt0();
  wg_barrier();
  if (rem > 0) {
    // The last, partial block, into stage 0.
    for (int cell = tid; cell < 512 * 8; cell += CF::NT) {
      const bool is_a = cell < 256 * 8;
      const int r = (cell / 8) & 255, c = cell % 8;
      int64_t row = (is_a ? m0 : n0) + r;
      const int64_t last = (is_a ? a.M : a.N) - 1;
      if (row > last) row = last;
      const char* p = (is_a ? a.A + row * a.lda : a.B + row * a.ldb) + (int64_t)nf * 128 + 16 * c;
      *reinterpret_cast<u32x4*>(smem + (is_a ? CF::A_AT : CF::B_AT) + r * 128 + ((c ^ f16r(r)) * 16)) =
          16 * c < rem ? load16(p) : zero4();
    }
    {
      const bool is_a = tid < 256;
      int64_t row = (is_a ? m0 : n0) + (tid & 255);
      const int64_t last = (is_a ? a.M : a.N) - 1;
      if (row > last) row = last;
      *reinterpret_cast<float*>(smem + CF::S_AT + tid * 4) =
          is_a ? a.SA[row * a.sa_m + nf * a.sa_k] : a.SB[(row >> a.shift) * a.sb_n + nf * a.sb_k];
    }
    __syncthreads();
    const float sbv = *reinterpret_cast<const float*>(sb) * kF8sUp;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      fm[j] = mask_block(read_a(0, j), g, rem);
      s[j] = *reinterpret_cast<const float*>(sa + j * 64) * sbv;
    }
#pragma unroll
    for (int i = 0; i < CF::FN; ++i) {
      const i32x8 fb = mask_block(read_b(0, i), g, rem);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = mfma_f8_block<FA, FB>(fb, fm[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(d[j][e], s[j], acc[i][j][e]);
    }
    wait_lgkmcnt0();
    wg_barrier();
  }
  uint32_t odd[4];
  const bool again = f8s_bring_down(acc, odd);
  // Through LDS, so that each store instruction writes four whole rows of the
  // wave's block (store_staged_block): a lane's 4 columns are half a chunk.
  char* const stage = smem + wave * (CF::WTM * CF::WTN * 2);
#pragma unroll
  for (int i = 0; i < CF::FN; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = j * 16 + lr, c = 2 * i + (g >> 1);
      *reinterpret_cast<u32x2*>(stage + r * 256 + ((c ^ (r & 15)) << 4) + 8 * (g & 1)) =
          u32x2{pack_out2<DT>(acc[i][j][0], acc[i][j][1]), pack_out2<DT>(acc[i][j][2], acc[i][j][3])};
    }
  const int64_t mw = m0 + wm * CF::WTM, nw = n0 + wn * CF::WTN;
  store_staged_block<CF::WTM, CF::WTN * 2>((char*)a.C + (mw * a.ldc + nw) * 2, a.ldc * 2, a.M - mw, (a.N - nw) * 2, stage, lane);
  if (again) f8s_store_again<FA, FB, false, CF::FN, CF::FM>(mw, nw, odd, lane);
}

}  // namespace gemmf16
