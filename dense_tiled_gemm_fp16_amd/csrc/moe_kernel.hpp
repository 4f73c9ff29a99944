// A mixture-of-experts layer for a few tokens in two kernels (gfx950).
//
// The weights of the experts that the tokens chose are all the time: they are
// read once, by the loops of strip_kernel.hpp, and everything else (routing,
// activation, weighted sum) happens around those loops so that nothing but
// the small activation array goes through memory between the two launches.
//
// Routing without a kernel of its own.  Expert e belongs to token t when
// fewer than top_k experts beat it: larger logit, or an equal one at a lower
// index.  That is a count over one row of logits, a ballot per 64 experts, so
// every workgroup of the first kernel finds the tokens of its expert by
// itself.  The rank (the count) is at the same time the expert's slot among
// the token's top_k, so results go to row t * top_k + rank of an array whose
// rows need no sorting or prefix sums.
//
//   moe_up    workgroup -> (expert, 16 rows of I): gate and up strips of
//             16 rows each over all of H, the waves splitting H; sums, silu(g)
//             u, two 16-bit parts per value into row (token, slot).  With
//             fewer (token, slot) pairs than experts, a workgroup is tied to a
//             pair instead, and only the first pair of an expert goes on.  The
//             workgroups of the first strip also write the pair's expert and
//             its softmax weight.
//   moe_down  workgroup -> 16 columns of Y, all experts: the waves share the
//             (expert, chunk of I) sequence evenly, each adds p * (sums) into
//             its own [T, 16] accumulators in LDS at every expert's end, and
//             the waves' accumulators are added in order.  So the weighted sum
//             over experts needs no atomics and no further pass.
#pragma once

#include "strip_kernel.hpp"

namespace gemmf16 {

constexpr int kMoeTokens = 64, kMoeExperts = 512, kMoeTopK = 16;
constexpr int kMoePairs = kMoeTokens * kMoeTopK;

struct MoeArgs {
  const char* x;
  int64_t ldx;                 // bytes
  const void* logits;
  int64_t ldl;                 // elements
  const char *w1, *w2;
  int64_t w1_e, w1_n, w2_e, w2_n;   // bytes
  const uint8_t *s1, *s2;
  int64_t s1_e, s1_n, s2_e, s2_n;
  uint16_t* y;
  int64_t ldy;
  char* act;                   // [T top_k][ip] 16-bit, then the second parts
  int64_t act_row, act_part;   // bytes of a row, of a part
  int32_t* tab_e;              // [T top_k] expert, -1 none
  float* tab_p;                // its softmax over all experts
  int64_t H, I;
  int32_t T, E, k, fmt_l, by_pair, renormalize;
};

// Logit as an integer of the same order: NaN above all, both zeros equal.
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (l != l) return 0xFFFFFFFFu;
  const uint32_t b = __builtin_bit_cast(uint32_t, l == 0.0f ? 0.0f : l);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float load_logit(const MoeArgs& a, int t, int e) {
  const int64_t i = t * a.ldl + e;
  if (a.fmt_l == 2) return ((const float*)a.logits)[i];
  const uint16_t h = ((const uint16_t*)a.logits)[i];
  return a.fmt_l == 0 ? cvt_in<DT_F16>(h) : cvt_in<DT_BF16>(h);
}

// Experts of token t that come before e (a whole wave).
__device__ __forceinline__ int logit_rank(const MoeArgs& a, int t, int e, uint32_t ke, int lane) {
  int n = 0;
  for (int j0 = 0; j0 < a.E; j0 += 64) {
    const int j = j0 + lane;
    bool before = false;
    if (j < a.E) {
      const uint32_t kj = logit_key(load_logit(a, t, j));
      before = kj > ke || (kj == ke && j < e);
    }
    n += __popcll(__ballot(before));
  }
  return n;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// exp(L[t,e]) / sum_j exp(L[t,j]) (a whole wave).
__device__ __forceinline__ float softmax_weight(const MoeArgs& a, int t, int e, int lane) {
  float m = -__builtin_inff();
  for (int j = lane; j < a.E; j += 64) m = fmaxf(m, load_logit(a, t, j));
  m = wave_max(m);
  float s = 0.0f;
  for (int j = lane; j < a.E; j += 64) s += expf(load_logit(a, t, j) - m);
  s = wave_sum(s);
  return expf(load_logit(a, t, e) - m) / s;
}

// silu(g) u as two parts of the format the down product takes.
template <bool F16>
__device__ __forceinline__ void split_parts(float v, uint16_t& hi, uint16_t& lo) {
  constexpr int DT = F16 ? DT_F16 : DT_BF16;
  hi = cvt_out<DT>(v);
  const float r = v - cvt_in<DT>(hi);
  lo = cvt_out<DT>(r == r && fabsf(r) <= fabsf(v) ? r : 0.0f);   // nothing beside an infinity or a NaN
}

struct MoeUpShared {
  union {
    f32x4 part[kStripWaves * 2 * 4 * 64];
    uint32_t key[kMoeExperts];
  };
  int rank[kMoeTokens];     // slot of the expert in the token's choice, -1 not chosen
  int list[kMoeTokens];     // the expert's tokens
  int count, found;
};

template <int WF, int DT, int MT, int UC>
__device__ __forceinline__ void moe_up_tiles(const MoeArgs& a, MoeUpShared& sh, int e, int64_t i0, int lane,
                                             int wave) {
  using S = Strip<WF, DT == DT_F16 ? SX_F16 : SX_BF16, 2, MT, UC>;
  const int m = sh.count;
  S s;
  s.xp = 0;
  int64_t row = i0 + (lane & 15);
  if (row >= a.I) row = a.I - 1;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    s.w[h] = a.w1 + e * a.w1_e + (h * a.I + row) * a.w1_n;
    s.ws[h] = a.s1 + e * a.s1_e + (h * a.I + row) * a.s1_n;
  }
  f32x4 acc[2][MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int p = 16 * t + (lane & 15);
    s.x[t] = a.x + sh.list[p < m ? p : m - 1] * a.ldx;
    s.xs[t] = nullptr;
    acc[0][t] = acc[1][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const int64_t nc = S::chunks(a.H);
  s.run(acc, nc * wave / kStripWaves, nc * (wave + 1) / kStripWaves, a.H, lane);
  constexpr int TILES = 2 * MT;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int t = 0; t < MT; ++t) sh.part[(wave * TILES + h * MT + t) * 64 + lane] = acc[h][t];
  __syncthreads();
  if (wave < MT) {
    const f32x4 gate = sum_waves<kStripWaves, TILES>(sh.part, wave, lane);
    const f32x4 up = sum_waves<kStripWaves, TILES>(sh.part, MT + wave, lane);
    const int p = 16 * wave + (lane & 15);
    const int64_t i = i0 + 4 * (lane >> 4);
    if (p < m && i < a.I) {       // rows hold a multiple of 8 values: all four fit
      const int t = sh.list[p];
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        split_parts<WF == SW_F16>(gate[r] / (1.0f + expf(-gate[r])) * up[r], hi[r], lo[r]);
      char* q = a.act + (t * a.k + sh.rank[t]) * a.act_row + 2 * i;
      __builtin_memcpy(q, hi, 8);
      __builtin_memcpy(q + a.act_part, lo, 8);
    }
  }
}

// Grid (strips of 16 rows of I, experts or pairs).  DT: format of X.
template <int WF, int DT>
__global__ __launch_bounds__(64 * kStripWaves) void moe_up_kernel(MoeArgs a) {
  __shared__ MoeUpShared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.y;
  int e = slot;
  if (a.by_pair) {
    // The expert of rank slot % k of token slot / k.
    const int t0 = slot / a.k, r0 = slot - t0 * a.k;
    for (int j = tid; j < a.E; j += 64 * kStripWaves) sh.key[j] = logit_key(load_logit(a, t0, j));
    __syncthreads();
    for (int c = tid; c < a.E; c += 64 * kStripWaves) {
      const uint32_t kc = sh.key[c];
      int n = 0;
      for (int j = 0; j < a.E; ++j) n += (sh.key[j] > kc || (sh.key[j] == kc && j < c)) ? 1 : 0;
      if (n == r0) sh.found = c;   // ranks are a permutation: exactly one
    }
    __syncthreads();
    e = __builtin_amdgcn_readfirstlane(sh.found);
    if (sh.key[e] == kKeyMinusInf) {   // the token has fewer than top_k experts
      if (blockIdx.x == 0 && tid == 0) {
        a.tab_e[slot] = -1;
        a.tab_p[slot] = 0.0f;
      }
      return;
    }
    __syncthreads();
  }
  const bool writes = blockIdx.x == 0;
  for (int t = wave; t < a.T; t += kStripWaves) {
    const float l = load_logit(a, t, e);
    const uint32_t ke = logit_key(l);
    const int r = logit_rank(a, t, e, ke, lane);
    const bool none = ke == kKeyMinusInf;
    if (lane == 0) sh.rank[t] = r < a.k && !none ? r : -1;
    if (writes && !a.by_pair && r < a.k && none && lane == 0) {
      a.tab_e[t * a.k + r] = -1;
      a.tab_p[t * a.k + r] = 0.0f;
    }
  }
  __syncthreads();
  if (wave == 0) {
    const bool mine = lane < a.T && sh.rank[lane] >= 0;
    const uint64_t all = __ballot(mine);
    if (mine) sh.list[__popcll(all & ((1ull << lane) - 1))] = lane;
    if (lane == 0) sh.count = __popcll(all);
  }
  __syncthreads();
  const int m = __builtin_amdgcn_readfirstlane(sh.count);
  if (m == 0) return;
  if (a.by_pair && __builtin_amdgcn_readfirstlane(sh.list[0]) != slot / a.k) return;
  if (writes) {
    for (int i = wave; i < m; i += kStripWaves) {
      const int t = sh.list[i];
      const float p = softmax_weight(a, t, e, lane);
      if (lane == 0) {
        a.tab_e[t * a.k + sh.rank[t]] = e;
        a.tab_p[t * a.k + sh.rank[t]] = p;
      }
    }
  }
  const int64_t i0 = (int64_t)blockIdx.x * 16;
  if (m <= 16)
    moe_up_tiles<WF, DT, 1, WF == SW_MX4 ? 2 : 4>(a, sh, e, i0, lane, wave);
  else if (m <= 32)
    moe_up_tiles<WF, DT, 2, WF == SW_MX4 ? 1 : 4>(a, sh, e, i0, lane, wave);
  else
    moe_up_tiles<WF, DT, 4, WF == SW_MX4 ? 1 : 2>(a, sh, e, i0, lane, wave);
}

struct MoeDownShared {
  float own[kStripWaves][kMoeTokens][16];
  uint32_t mask[kMoeExperts][2];     // tokens of an expert
  uint16_t active[kMoeExperts], place[kMoeExperts];
  uint16_t start[kMoeExperts + 1];
  uint32_t rows[kMoePairs];          // token << 16 | pair, by expert
  int32_t expert[kMoePairs];
  float prob[kMoePairs];
  int n_active;
};

// p * (W2[e] rows h0 .. h0+15) (act rows of e) over chunks [c0, c1), into this
// wave's accumulators.
template <int WF, int MT, int UC>
__device__ __forceinline__ void moe_down_segment(const MoeArgs& a, MoeDownShared& sh, int e, int first, int m,
                                                 int64_t h0, int64_t c0, int64_t c1, int lane, int wave) {
  using S = Strip<WF, WF == SW_F16 ? SX_F16P : SX_BF16P, 1, MT, UC>;
  S s;
  s.xp = a.act_part;
  int64_t row = h0 + (lane & 15);
  if (row >= a.H) row = a.H - 1;
  s.w[0] = a.w2 + e * a.w2_e + row * a.w2_n;
  s.ws[0] = a.s2 + e * a.s2_e + row * a.s2_n;
  f32x4 acc[1][MT];
  uint32_t who[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int p = 16 * t + (lane & 15);
    who[t] = sh.rows[first + (p < m ? p : m - 1)];
    s.x[t] = a.act + (int64_t)(who[t] & 0xFFFFu) * a.act_row;
    s.xs[t] = nullptr;
    acc[0][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  s.run(acc, c0, c1, a.I, lane);
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (16 * t + (lane & 15) < m) {
      const float p = sh.prob[who[t] & 0xFFFFu];
      float* q = &sh.own[wave][who[t] >> 16][4 * (lane >> 4)];
#pragma unroll
      for (int r = 0; r < 4; ++r) q[r] += p * acc[0][t][r];
    }
  }
}

template <int WF, int DT>
__global__ __launch_bounds__(64 * kStripWaves) void moe_down_kernel(MoeArgs a) {
  __shared__ MoeDownShared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int NT = 64 * kStripWaves;
  const int pairs = a.T * a.k;
  for (int i = tid; i < a.E; i += NT) sh.mask[i][0] = sh.mask[i][1] = 0;
  for (int i = tid; i < pairs; i += NT) {
    sh.expert[i] = a.tab_e[i];
    sh.prob[i] = a.tab_p[i];
  }
  for (int i = lane; i < a.T * 16; i += 64) sh.own[wave][i / 16][i % 16] = 0.0f;
  __syncthreads();
  for (int i = tid; i < pairs; i += NT) {
    const int t = i / a.k;
    if (sh.expert[i] >= 0) atomicOr(&sh.mask[sh.expert[i]][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  if (wave == 0) {
    // The experts in use, in order, and where their rows start.
    int n = 0, at = 0;
    for (int j0 = 0; j0 < a.E; j0 += 64) {
      const int j = j0 + lane;
      const int c = j < a.E ? __popc(sh.mask[j][0]) + __popc(sh.mask[j][1]) : 0;
      int upto = c;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
      }
      const uint64_t used = __ballot(c > 0);
      if (c > 0) {
        const int i = n + __popcll(used & ((1ull << lane) - 1));
        sh.active[i] = (uint16_t)j;
        sh.place[j] = (uint16_t)i;
        sh.start[i] = (uint16_t)(at + upto - c);
      }
      n += __popcll(used);
      at += __shfl(upto, 63);
    }
    if (lane == 0) {
      sh.start[n] = (uint16_t)at;
      sh.n_active = n;
    }
  }
  __syncthreads();
  float prob[(kMoePairs + NT - 1) / NT];
#pragma unroll
  for (int q = 0; q < (kMoePairs + NT - 1) / NT; ++q) {
    const int i = tid + q * NT;
    if (i >= pairs || sh.expert[i] < 0) continue;
    const int t = i / a.k, e = sh.expert[i];
    const uint64_t mask = (uint64_t)sh.mask[e][0] | ((uint64_t)sh.mask[e][1] << 32);
    sh.rows[sh.start[sh.place[e]] + __popcll(mask & ((1ull << t) - 1))] = (uint32_t)t << 16 | (uint32_t)i;
    prob[q] = sh.prob[i];
    if (a.renormalize) {
      float s = 0.0f;
      for (int j = 0; j < a.k; ++j) s += sh.prob[t * a.k + j];
      prob[q] /= s;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < (kMoePairs + NT - 1) / NT; ++q) {
    const int i = tid + q * NT;
    if (i < pairs && sh.expert[i] >= 0) sh.prob[i] = prob[q];
  }
  __syncthreads();

  const int64_t h0 = (int64_t)blockIdx.x * 16;
  constexpr int CK = WF == SW_MX4 ? 128 : 32;
  const int cpe = (int)((a.I + CK - 1) / CK), n = __builtin_amdgcn_readfirstlane(sh.n_active);
  const int64_t units = (int64_t)n * cpe;
  int64_t u = units * wave / kStripWaves;
  const int64_t u1 = units * (wave + 1) / kStripWaves;
  while (u < u1) {
    const int i = (int)(u / cpe), c0 = (int)(u - (int64_t)i * cpe);
    const int c1 = (int)(c0 + (u1 - u) < cpe ? c0 + (u1 - u) : cpe);
    const int e = __builtin_amdgcn_readfirstlane(sh.active[i]);
    const int first = __builtin_amdgcn_readfirstlane(sh.start[i]);
    const int m = __builtin_amdgcn_readfirstlane(sh.start[i + 1]) - first;
    if (m <= 16)
      moe_down_segment<WF, 1, WF == SW_MX4 ? 2 : 4>(a, sh, e, first, m, h0, c0, c1, lane, wave);
    else if (m <= 32)
      moe_down_segment<WF, 2, WF == SW_MX4 ? 1 : 4>(a, sh, e, first, m, h0, c0, c1, lane, wave);
    else
      moe_down_segment<WF, 4, WF == SW_MX4 ? 1 : 2>(a, sh, e, first, m, h0, c0, c1, lane, wave);
    u += c1 - c0;
  }
  __syncthreads();
  for (int i = tid; i < a.T * 4; i += NT) {
    const int t = i >> 2, g = i & 3;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kStripWaves; ++w)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] += sh.own[w][t][4 * g + r];
    const int64_t h = h0 + 4 * g;
    uint16_t* y = a.y + t * a.ldy + h;
    uint16_t o[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = cvt_out<DT>(s[r]);
    if (h + 4 <= a.H) {
      __builtin_memcpy(y, o, 8);
    } else {
      for (int r = 0; r < 4 && h + r < a.H; ++r) y[r] = o[r];
    }
  }
}

}  // namespace gemmf16
