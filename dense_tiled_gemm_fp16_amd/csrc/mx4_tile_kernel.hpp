// Product of two MX FP4 matrices by 256 x 256 tiles (gfx950):
// C[m,n] = sum over blocks of sA sB sum over the block's k of a b.
//
// The matrix core's rate bounds it: v_mfma_scale_f32_32x32x64_f8f6f4 takes 64 k
// of 4-bit codes with a scale per row and block, four times the binary16
// instruction's work per cycle, so the tile has to bring 512 rows x 64 bytes
// into LDS in the time of 16 such instructions per wave.  The skeleton is that
// of the FP8 tile: 8 waves of 64 x 128, LDS-DMA without staging registers, two
// wave groups one phase apart, one reading fragments and issuing DMA while the
// other's matrix instructions run, raw barriers and counted waits.
//
//   LDS   4 stages of 128 k: 256 A rows and 256 B rows of 64 bytes (16-byte
//         chunk c of row r in slot c ^ fa(r)), and one dword of four scales
//         for each of the 512 rows.  The loads of step t + 3 are issued in step
//         t, into the stage that every wave has finished reading.
//   k     A lane of group g = lane / 32 reads chunks 2 g and 2 g + 1 of its
//         row, two blocks of 32 k: the operands of the step's two
//         instructions per 32 x 32 block, the same for A and B.  Their scales
//         are bytes 2 g and 2 g + 1 of the row's dword, shifted down once, then
//         picked by the instruction's byte select.
//
// Scales as they lie (one byte per block, rows far apart) would cost a line
// per row and step, as much of the load path as the codes.  A small kernel
// first transposes both scale arrays to [steps][rows] dwords, so that a step's
// scales are 2 KiB of consecutive bytes: eight 256-byte DMA instructions.
//
// Measured: 32768 x 2048 x 7168 in 272 us after the quantiser (median of a kernel
// trace, the least 254), 253 with the scales' kernel call after call in a graph
// (3.8 PFLOP/s; binary16's main kernel 1.3), 228 to 240 on another machine; 4096^3
// 42 us (3.3).  The scales take 7 and 4 us of it.  Four waves of 128 x 128, with two
// thirds of the LDS reads, took 264 us beside 243 in one run: it is not the LDS but
// the clock that the matrix core's power leaves.
//
// k past K: the last step, if K is no multiple of 128, is filled through
// registers, codes of A past K zeroed.
#pragma once

#include "dma_a128_kernel.hpp"
#include "mx4_common.hpp"

namespace gemmf16 {

struct Mx4Cfg {
  static constexpr int BM = 256, BN = 256, BK = 64;   // BK in bytes: 128 k
  static constexpr int WAVES_M = 4, WAVES_N = 2, NW = 8, NT = 512;
  static constexpr int WTM = 64, WTN = 128, FM = 2, FN = 4;
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, S_BYTES = (BM + BN) * 4;
  static constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES, STAGES = 4;
  static constexpr int LDS = STAGES * STAGE;
  static constexpr int DMA_A = A_BYTES / 1024 / NW, DMA_B = B_BYTES / 1024 / NW;
  static constexpr int DMA_PER_STEP = DMA_A + DMA_B + 1;
  static_assert(LDS <= 160 * 1024, "LDS budget");
  static_assert(S_BYTES == NW * 256, "one scale instruction per wave and step");
};

struct Mx4TileArgs {
  KArgs k;               // A, lda_m, B, ldb_n (bytes), C, ldc, M, N, K, GM, GN, panel
  const uint32_t* sa;    // [ceil(K/128)][sa_rows] dwords of four scales
  int64_t sa_rows;       // M up to a multiple of 256
  const uint32_t* sb;
  int64_t sb_rows;
};

// Scale rows [R][Kb] bytes (row stride ld) -> dst[t][r] = scales 4 t .. 4 t + 3
// of row r; 2^0 past the end.  A and B in one launch: blockIdx.z picks.
struct Mx4ScaleArgs {
  const uint8_t* src[2];
  int64_t ld[2], rows[2], padded[2];
  uint32_t* dst[2];
  int64_t Kb, steps;
};

__global__ __launch_bounds__(256) void mx4_scales_kernel(Mx4ScaleArgs a) {
  // A block takes 64 rows x 16 steps: 64 bytes of each row, read four steps
  // to a lane, written as runs of 64 dwords.
  __shared__ uint32_t tile[16][65];
  const int w = blockIdx.z;
  const int64_t r0 = (int64_t)blockIdx.x * 64, t0 = (int64_t)blockIdx.y * 16;
  if (r0 >= a.padded[w]) return;
  const int r = threadIdx.x >> 2, q = threadIdx.x & 3;
  const int64_t row = r0 + r, b0 = 4 * (t0 + 4 * q);
  const uint8_t* p = a.src[w] + row * a.ld[w] + b0;
  if (row < a.rows[w] && b0 + 16 <= a.Kb) {
    const u32x4 v = load16(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) tile[4 * q + i][r] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t d = 0x7F7F7F7Fu;
      if (row < a.rows[w])
        for (int j = 0; j < 4; ++j)
          if (b0 + 4 * i + j < a.Kb) d = (d & ~(0xFFu << (8 * j))) | (uint32_t)p[4 * i + j] << (8 * j);
      tile[4 * q + i][r] = d;
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = (threadIdx.x >> 6) + 4 * i;
    if (t0 + t < a.steps && r0 + lane < a.padded[w])
      a.dst[w][(t0 + t) * a.padded[w] + r0 + lane] = tile[t][lane];
  }
}

struct Mx4Frag {
  u32x4 c[2];       // blocks 2 g and 2 g + 1 of a row
  uint32_t s;       // their scales in bytes 0 and 1
};

// Row r of a stage's operand; `st` its codes, `sc` its scales.
__device__ __forceinline__ Mx4Frag read_mx4(const char* st, const char* sc, int r, int g) {
  Mx4Frag f;
  const char* row = st + r * 64;
  f.c[0] = *reinterpret_cast<const u32x4*>(row + (((2 * g) ^ fa(r)) * 16));
  f.c[1] = *reinterpret_cast<const u32x4*>(row + (((2 * g + 1) ^ fa(r)) * 16));
  f.s = *reinterpret_cast<const uint32_t*>(sc + r * 4) >> (16 * g);
  return f;
}

__device__ __forceinline__ i32x8 low4(u32x4 v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// Both instructions of a 32 x 32 block; first operand the B block.
__device__ __forceinline__ f32x16 mma_mx4(const Mx4Frag& b, const Mx4Frag& a, f32x16 c) {
  c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(low4(b.c[0]), low4(a.c[0]), c, 4, 4, 0, (int)b.s, 0,
                                                      (int)a.s);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(low4(b.c[1]), low4(a.c[1]), c, 4, 4, 1, (int)b.s, 1,
                                                         (int)a.s);
}

template <int DT>
__global__ __launch_bounds__(Mx4Cfg::NT) void mx4_tile_kernel(Mx4TileArgs args) {
  using CF = Mx4Cfg;
  const KArgs& a = args.k;
  __shared__ __attribute__((aligned(1024))) char smem[CF::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / CF::WAVES_N, wn = wave % CF::WAVES_N;
  const int lr = lane % 32, g = lane / 32;

  int64_t pm, pn;
  raster_tile(blockIdx.x, a.GM, a.GN, a.panel, pm, pn);
  const int64_t m0 = pm * CF::BM, n0 = pn * CF::BN;

  // The DMA helpers count 16-bit units: half the byte strides.
  BSourceS<CF::DMA_A, true> sa;
  BSourceS<CF::DMA_B, true> sb;
  sa.init(a.A, a.lda_m / 2, 1, a.M, m0, 0, wave, lane);
  sb.init(a.B, a.ldb_n / 2, 1, a.N, n0, 0, wave, lane);
  // Scale instruction of this wave: rows 64 w .. of A, then of B.
  const bool sw_a = wave < CF::BM / 64;
  const char* ps = uniform_ptr(sw_a ? (const char*)(args.sa + m0 + 64 * wave)
                                    : (const char*)(args.sb + n0 + 64 * (wave - CF::BM / 64)));
  const int64_t s_step = 4 * (sw_a ? args.sa_rows : args.sb_rows);
  const uint32_t s_off = 4 * lane;

  f32x16 acc[CF::FN][CF::FM];
#pragma unroll
  for (int i = 0; i < CF::FN; ++i)
#pragma unroll
    for (int j = 0; j < CF::FM; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  auto stage = [&](int t) { return smem + (t & (CF::STAGES - 1)) * CF::STAGE; };
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  auto issue = [&](int t, const char* pa, const char* pb, const char* pc) {
    const uint32_t st = lds0 + (t & (CF::STAGES - 1)) * CF::STAGE;
    sa.issue_batch_at(st + CF::DMA_A * wave * 1024, pa);
    sb.issue_batch_at(st + CF::A_BYTES + CF::DMA_B * wave * 1024, pb);
    dma4s(s_off, pc, st + CF::A_BYTES + CF::B_BYTES + wave * 256);
  };
  auto read_a = [&](int t, int j) {
    const char* st = stage(t);
    return read_mx4(st, st + CF::A_BYTES + CF::B_BYTES, wm * CF::WTM + j * 32 + lr, g);
  };
  auto read_b = [&](int t, int i) {
    const char* st = stage(t);
    return read_mx4(st + CF::A_BYTES, st + CF::A_BYTES + CF::B_BYTES + CF::BM * 4, wn * CF::WTN + i * 32 + lr, g);
  };

  const int nf = (int)(a.K / 128);       // whole steps
  const int rem = (int)(a.K - (int64_t)nf * 128);
  Mx4Frag fb[CF::FN], fm[CF::FM];

  if (nf > 0) {
    const bool g1 = wave >= CF::NW / 2;
    auto at = [&](int t) { return t < nf ? t : nf - 1; };
#pragma unroll
    for (int t = 0; t < CF::STAGES - 1; ++t)
      issue(t, sa.base + at(t) * sa.step, sb.base + at(t) * sb.step, ps + at(t) * s_step);
    wait_vmcnt<CF::DMA_PER_STEP>();      // steps 0 and 1 landed
    wg_barrier();
    fb[0] = read_b(0, 0);
    fb[1] = read_b(0, 1);
    if (g1) wg_barrier();

    const char* pa = sa.base + at(3) * sa.step;
    const char* pb = sb.base + at(3) * sb.step;
    const char* pc = ps + at(3) * s_step;
    for (int t = 0; t < nf; ++t) {
      // Memory phase: this step's A blocks and B blocks 2 and 3, DMA of step
      // t + 3 (into the stage of step t - 1, which no wave reads any more; past
      // the end it re-loads the last step).
      fm[0] = read_a(t, 0);
      fm[1] = read_a(t, 1);
      fb[2] = read_b(t, 2);
      fb[3] = read_b(t, 3);
      issue(t + 3, pa, pb, pc);
      if (t + 4 < nf) {
        pa += sa.step;
        pb += sb.step;
        pc += s_step;
      }
      wait_lgkmcnt0();
      __builtin_amdgcn_sched_barrier(0);
      // Compute phase; B blocks 0 and 1 of step t + 1 are read under its
      // second half (on the last step, unused bytes of a free stage).
      __builtin_amdgcn_s_setprio(1);
      acc[0][0] = mma_mx4(fb[0], fm[0], acc[0][0]);
      wg_barrier();
      __builtin_amdgcn_sched_barrier(0);
      acc[0][1] = mma_mx4(fb[0], fm[1], acc[0][1]);
      acc[1][0] = mma_mx4(fb[1], fm[0], acc[1][0]);
      acc[1][1] = mma_mx4(fb[1], fm[1], acc[1][1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 2; i < CF::FN; ++i)
#pragma unroll
        for (int j = 0; j < CF::FM; ++j) {
          acc[i][j] = mma_mx4(fb[i], fm[j], acc[i][j]);
          if (j == 0) fb[i - 2] = read_b(t + 1, i - 2);
          __builtin_amdgcn_sched_barrier(0);
        }
      wait_vmcnt<CF::DMA_PER_STEP>();    // step t + 2 landed
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(0);
      wg_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!g1) wg_barrier();   // pairs with group 1's extra first barrier
    wait_vmcnt<0>();         // no LDS transfer may still be in flight past this point
  }
  if (rem > 0) {
    // The last, partial step, into stage nf (free after the last barrier).
    wg_barrier();
    char* st = stage(nf);
    for (int cell = tid; cell < (CF::BM + CF::BN) * 4; cell += CF::NT) {
      const bool is_a = cell < CF::BM * 4;
      const int r = (is_a ? cell : cell - CF::BM * 4) / 4, c = cell % 4;
      int64_t row = (is_a ? m0 : n0) + r;
      const int64_t last = (is_a ? a.M : a.N) - 1;
      if (row > last) row = last;
      const char* p = (const char*)(is_a ? a.A : a.B) + row * (is_a ? a.lda_m : a.ldb_n) + (int64_t)nf * 64 + 16 * c;
      const int left = rem - 32 * c;
      u32x4 v = left > 0 ? load16(p) : zero4();
      if (is_a && left > 0 && left < 32) v = mask_codes(v, left);
      *reinterpret_cast<u32x4*>(st + (is_a ? 0 : CF::A_BYTES) + r * 64 + ((c ^ fa(r)) * 16)) = v;
    }
    {
      const uint32_t v = tid < CF::BM ? args.sa[(int64_t)nf * args.sa_rows + m0 + tid]
                                      : args.sb[(int64_t)nf * args.sb_rows + n0 + tid - CF::BM];
      *reinterpret_cast<uint32_t*>(st + CF::A_BYTES + CF::B_BYTES + tid * 4) = v;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < CF::FN; ++i) fb[i] = read_b(nf, i);
#pragma unroll
    for (int j = 0; j < CF::FM; ++j) fm[j] = read_a(nf, j);
#pragma unroll
    for (int i = 0; i < CF::FN; ++i)
#pragma unroll
      for (int j = 0; j < CF::FM; ++j) acc[i][j] = mma_mx4(fb[i], fm[j], acc[i][j]);
  }
  wait_lgkmcnt0();
  wg_barrier();
  store_tile_staged<CF, DT>(a, acc, smem, m0, n0, wave, wm, wn, lane);
}

}  // namespace gemmf16
