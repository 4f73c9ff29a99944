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
//   LDS    S stages of 128 k: BM rows of A and BN rows of B, 128 bytes each,
//          16-byte chunk c of row r in slot c ^ f8(r), and a dword of scale for
//          each row.  All comes by LDS-DMA (8 whole lines an instruction; the
//          scales as one dword a lane, so that any strides will do): step t + S
//          - 1 is issued into the stage of step t - 1 behind the one barrier of
//          step t.
//   k      a lane of group g = lane / 16 takes chunks g and g + 4 of its row,
//          for A and B alike: any assignment of k to bytes that both share is
//          the product.
//   sums   the first operand is B: a lane holds columns 4 (lane / 16) .. + 3 of
//          row lane % 16 of C, so one multiplication gives the scale of a row
//          and a block of columns, and 8 or 16 consecutive bytes are stored.
//
// K past the last whole block is filled through registers with zeros on both
// sides; rows past M or N read the last valid row and are never stored.
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
  int32_t splits;           // parts of K; > 1: float32 sums to W[part][M][N]
  int64_t part_steps;       // steps of a part
  float* W;
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
  static constexpr int DMA_A = A_BYTES / 1024, DMA_B = B_BYTES / 1024;   // instructions of the workgroup
  static constexpr int DI = (DMA_A + DMA_B) / NW;                        // per wave
  static constexpr int PER_STEP = DI + SI;
  static_assert((DMA_A + DMA_B) % NW == 0 && TM % 16 == 0 && TN % 16 == 0 && 128 % TN == 0, "shape");
  static_assert(LDS <= 160 * 1024, "LDS budget");
};

// One 256-byte DMA: lane l's dword at base + off lands at LDS lds + 4 l.
__device__ __forceinline__ void dma4_any(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds), "v"(p)
               : "memory", "m0");
}
__device__ __forceinline__ void dma16_any(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(p)
               : "memory", "m0");
}

template <int FA, int FB>
__device__ __forceinline__ f32x4 mfma_f8_block(const i32x8& b, const i32x8& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, FB, FA, 0, 0, 0, 0);
}

// Chunks g and g + 4 of row r of an operand's stage.
__device__ __forceinline__ i32x8 read_f8_row(const char* st, int r, int g) {
  const char* row = st + r * 128;
  return join8(*reinterpret_cast<const u32x4*>(row + ((g ^ f8(r)) * 16)),
               *reinterpret_cast<const u32x4*>(row + (((g + 4) ^ f8(r)) * 16)));
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

template <class CF, int FA, int FB, bool ROWB>
__global__ __launch_bounds__(CF::NT) void f8s_tile_kernel(F8sArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[CF::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / CF::WN, wn = wave % CF::WN;
  const int lr = lane & 15, g = lane >> 4;

  int64_t pm, pn, w = blockIdx.x;
  int64_t part = 0;
  if (a.splits > 1) {
    part = w / (a.GM * a.GN);
    w -= part * (a.GM * a.GN);
  }
  raster_tile(w, a.GM, a.GN, a.panel, pm, pn);
  const int64_t m0 = pm * CF::BM, n0 = pn * CF::BN;
  const int64_t k0 = part * a.part_steps * 128;
  const int64_t ke = a.splits > 1 && k0 + a.part_steps * 128 < a.K ? k0 + a.part_steps * 128 : a.K;

  // This wave's DMA instructions of a step: DI of 8 rows, A's first, then SI of
  // 64 scales, A's first (the last may be one too many: it repeats B's rows).
  const char* src[CF::DI];
  const char* ssrc[CF::SI];
  int64_t sstep[CF::SI];
#pragma unroll
  for (int i = 0; i < CF::DI; ++i) {
    const int q = wave * CF::DI + i;
    const bool is_a = q < CF::DMA_A;
    const int r = (is_a ? q : q - CF::DMA_A) * 8 + lane / 8, c = (lane % 8) ^ f8(r);
    int64_t row = (is_a ? m0 : n0) + r;
    const int64_t last = (is_a ? a.M : a.N) - 1;
    if (row > last) row = last;
    src[i] = (is_a ? a.A + row * a.lda : a.B + row * a.ldb) + k0 + 16 * c;
  }
#pragma unroll
  for (int i = 0; i < CF::SI; ++i) {
    const int q = wave * CF::SI + i;
    const bool is_a = q < (CF::BM + 63) / 64;
    int64_t row = (is_a ? m0 + q * 64 : n0 + (q - (CF::BM + 63) / 64) * 64) + lane;
    const int64_t last = (is_a ? a.M : a.N) - 1;
    if (row > last) row = last;
    const int64_t b0 = k0 / 128;
    ssrc[i] = (const char*)(is_a ? a.SA + row * a.sa_m + b0 * a.sa_k : a.SB + (row >> a.shift) * a.sb_n + b0 * a.sb_k);
    sstep[i] = 4 * (is_a ? a.sa_k : a.sb_k);
  }

  f32x4 acc[CF::FN][CF::FM];
#pragma unroll
  for (int i = 0; i < CF::FN; ++i)
#pragma unroll
    for (int j = 0; j < CF::FM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  auto issue = [&](int64_t t, int slot) {
    const uint32_t st = lds0 + slot * CF::STAGE;
#pragma unroll
    for (int i = 0; i < CF::DI; ++i) dma16_any(src[i] + t * 128, st + (wave * CF::DI + i) * 1024);
#pragma unroll
    for (int i = 0; i < CF::SI; ++i)
      dma4_any(ssrc[i] + t * sstep[i], st + CF::A_BYTES + CF::B_BYTES + (wave * CF::SI + i) * 256);
  };
  auto compute = [&](int slot) {
    const char* st = smem + slot * CF::STAGE;
    const char* sc = st + CF::A_BYTES + CF::B_BYTES;
    i32x8 fm[CF::FM];
    float s[CF::FM];
    const float sb = ROWB ? 1.0f : *(const float*)(sc + CF::SB_AT + wn * CF::TN * 4);
#pragma unroll
    for (int j = 0; j < CF::FM; ++j) {
      fm[j] = read_f8_row(st, wm * CF::TM + j * 16 + lr, g);
      s[j] = *(const float*)(sc + (wm * CF::TM + j * 16 + lr) * 4) * sb;
    }
#pragma unroll
    for (int i = 0; i < CF::FN; ++i) {
      const i32x8 fb = read_f8_row(st + CF::A_BYTES, wn * CF::TN + i * 16 + lr, g);
      f32x4 sn{1.0f, 1.0f, 1.0f, 1.0f};
      if constexpr (ROWB) sn = *(const f32x4*)(sc + CF::SB_AT + (wn * CF::TN + i * 16 + 4 * g) * 4);
      f32x4 d[CF::FM];
#pragma unroll
      for (int j = 0; j < CF::FM; ++j) d[j] = mfma_f8_block<FA, FB>(fb, fm[j]);
#pragma unroll
      for (int j = 0; j < CF::FM; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_fmaf(ROWB ? d[j][e] * sn[e] : d[j][e], s[j], acc[i][j][e]);
    }
  };

  const int64_t nf = (ke - k0) / 128;
  const int rem = (int)((ke - k0) - nf * 128);
  auto at = [&](int64_t t) { return t < nf ? t : nf - 1; };
  if (nf > 0) {
#pragma unroll
    for (int t = 0; t < CF::STAGES - 1; ++t) issue(at(t), t);
    int slot = 0;
    for (int64_t t = 0; t < nf; ++t) {
      wait_vmcnt<(CF::STAGES - 2) * CF::PER_STEP>();    // this wave's part of step t landed,
      wait_lgkmcnt0();                                  // and its reads of step t - 1 returned
      wg_barrier();                                     // both of every wave's
      issue(at(t + CF::STAGES - 1), slot == 0 ? CF::STAGES - 1 : slot - 1);
      compute(slot);
      slot = slot == CF::STAGES - 1 ? 0 : slot + 1;
    }
    wait_vmcnt<0>();
  }
  wait_lgkmcnt0();
  wg_barrier();
  if (rem > 0) {
    // The last, partial block, into stage 0 (free after the barrier).
    for (int cell = tid; cell < (CF::BM + CF::BN) * 8; cell += CF::NT) {
      const bool is_a = cell < CF::BM * 8;
      const int r = (is_a ? cell : cell - CF::BM * 8) / 8, c = cell % 8;
      int64_t row = (is_a ? m0 : n0) + r;
      const int64_t last = (is_a ? a.M : a.N) - 1;
      if (row > last) row = last;
      const char* p = (is_a ? a.A + row * a.lda : a.B + row * a.ldb) + k0 + nf * 128 + 16 * c;
      *reinterpret_cast<u32x4*>(smem + (is_a ? 0 : CF::A_BYTES) + r * 128 + ((c ^ f8(r)) * 16)) =
          load_bytes(p, rem - 16 * c);
    }
    for (int r = tid; r < CF::BM + CF::BN; r += CF::NT) {
      const bool is_a = r < CF::BM;
      int64_t row = is_a ? m0 + r : n0 + r - CF::BM;
      const int64_t last = (is_a ? a.M : a.N) - 1;
      if (row > last) row = last;
      const int64_t b = k0 / 128 + nf;
      const float v = is_a ? a.SA[row * a.sa_m + b * a.sa_k] : a.SB[(row >> a.shift) * a.sb_n + b * a.sb_k];
      *reinterpret_cast<float*>(smem + CF::A_BYTES + CF::B_BYTES + (is_a ? 4 * r : CF::SB_AT + 4 * (r - CF::BM))) = v;
    }
    __syncthreads();
    compute(0);
  }

  void* const C = a.splits > 1 ? (void*)(a.W + part * a.M * a.N) : a.C;
  const int out = a.splits > 1 ? (int)F8S_F32 : a.out;
  const int64_t ldc = a.splits > 1 ? a.N : a.ldc;
#pragma unroll
  for (int j = 0; j < CF::FM; ++j) {
    const int64_t m = m0 + wm * CF::TM + j * 16 + lr;
#pragma unroll
    for (int i = 0; i < CF::FN; ++i) {
      const int64_t n = n0 + wn * CF::TN + i * 16 + 4 * g;
      if (m < a.M && n < a.N) store_out4(C, out, m * ldc + n, acc[i][j], a.N - n);
    }
  }
}

}  // namespace gemmf16
