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
//   moe_up    wave -> (expert, 16 rows of I, a part of H): gate and up strips
//             of 16 rows each; the parts of H meet in LDS; silu(g) u, two
//             16-bit parts per value, into row (token, slot).  The waves of a
//             workgroup are kMoeWaves / parts neighbouring strips times the
//             parts: as few parts as still fill the device, so that a wave
//             streams long rows and the workgroup's waves meet A in L1.  With
//             fewer (token, slot) pairs than experts, a workgroup is tied to a
//             pair instead, and only the first pair of an expert goes on.  The
//             workgroups of the first strips also write the pair's expert and
//             its softmax weight.
//   moe_down  workgroup -> 16 columns of Y, all experts: the waves share the
//             (expert, chunk of I) sequence evenly, loads running ahead across
//             experts, each adds p * (sums) into its own [T, 16] accumulators
//             in LDS at every expert's end, and the waves' accumulators are
//             added in order.  So the weighted sum over experts needs no
//             atomics and no further pass.
#pragma once

#include "strip_kernel.hpp"

namespace gemmf16 {

constexpr int kMoeTokens = 64, kMoeExperts = 512, kMoeTopK = 16;
constexpr int kMoePairs = kMoeTokens * kMoeTopK;
constexpr int kMoeWaves = 8;

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
  int32_t parts;               // of H, in moe_up: 1, 2, 4 or 8
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

template <int MT>
struct MoeUpShared {
  union {
    f32x4 part[kMoeWaves * 2 * MT * 64];
    uint32_t key[kMoeExperts];
  };
  int rank[kMoeTokens];     // slot of the expert in the token's choice, -1 not chosen
  int list[kMoeTokens];     // the expert's tokens
  int count, found;
};

template <int WF, int DT, int MT, int UC>
__device__ __forceinline__ void moe_up_tiles(const MoeArgs& a, MoeUpShared<MT>& sh, int e, int lane, int wave) {
  using S = Strip<WF, DT == DT_F16 ? SX_F16 : SX_BF16, 2, MT, UC>;
  constexpr int TILES = 2 * MT;
  const int m = __builtin_amdgcn_readfirstlane(sh.count), tiles = (m + 15) / 16;
  const int strips = kMoeWaves / a.parts;      // of this workgroup
  const int strip = wave / a.parts, part = wave - strip * a.parts;
  const int64_t i0 = ((int64_t)blockIdx.x * strips + strip) * 16;
  if (i0 < a.I) {
    typename S::WPtr w;
    typename S::XPtr x;
    x.part = 0;
    int64_t row = i0 + (lane & 15);
    if (row >= a.I) row = a.I - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w.w[h] = a.w1 + e * a.w1_e + (h * a.I + row) * a.w1_n;
      w.s[h] = a.s1 + e * a.s1_e + (h * a.I + row) * a.s1_n;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int p = 16 * t + (lane & 15);
      x.x[t] = a.x + sh.list[p < m ? p : m - 1] * a.ldx;
      x.s[t] = nullptr;
    }
    f32x4 acc[2][MT];
    S::clear(acc);
    const int64_t nc = S::chunks(a.H);
    S::run(acc, w, x, nc * part / a.parts, nc * (part + 1) / a.parts, a.H, lane >> 4, tiles == 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < MT; ++t) sh.part[(wave * TILES + h * MT + t) * 64 + lane] = acc[h][t];
  }
  __syncthreads();
  for (int j = wave; j < strips * tiles; j += kMoeWaves) {
    const int s = j / tiles, t = j - s * tiles;
    const f32x4* base = sh.part + s * a.parts * TILES * 64 + t * 64;
    const int p = 16 * t + (lane & 15);
    const int64_t i = ((int64_t)blockIdx.x * strips + s) * 16 + 4 * (lane >> 4);
    if (p < m && i < a.I) {       // rows hold a multiple of 8 values: all four fit
      const f32x4 gate = sum_waves(base, TILES * 64, a.parts, lane);
      const f32x4 up = sum_waves(base + MT * 64, TILES * 64, a.parts, lane);
      const int token = sh.list[p];
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        split_parts<WF == SW_F16>(gate[r] / (1.0f + expf(-gate[r])) * up[r], hi[r], lo[r]);
      char* q = a.act + (token * a.k + sh.rank[token]) * a.act_row + 2 * i;
      __builtin_memcpy(q, hi, 8);
      __builtin_memcpy(q + a.act_part, lo, 8);
    }
  }
}

// Grid (groups of strips of 16 rows of I, experts or pairs).  DT: format of X;
// MT: tiles of 16 tokens that T needs.
template <int WF, int DT, int MT>
__global__ __launch_bounds__(64 * kMoeWaves, MT < 2 ? 4 : 2) void moe_up_kernel(MoeArgs a) {
  __shared__ MoeUpShared<MT> sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.y;
  int e = slot;
  if (a.by_pair) {
    // The expert of rank slot % k of token slot / k.
    const int t0 = slot / a.k, r0 = slot - t0 * a.k;
    for (int j = tid; j < a.E; j += 64 * kMoeWaves) sh.key[j] = logit_key(load_logit(a, t0, j));
    __syncthreads();
    for (int c = tid; c < a.E; c += 64 * kMoeWaves) {
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
  for (int t = wave; t < a.T; t += kMoeWaves) {
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
    for (int i = wave; i < m; i += kMoeWaves) {
      const int t = sh.list[i];
      const float p = softmax_weight(a, t, e, lane);
      if (lane == 0) {
        a.tab_e[t * a.k + sh.rank[t]] = e;
        a.tab_p[t * a.k + sh.rank[t]] = p;
      }
    }
  }
  moe_up_tiles<WF, DT, MT, WF == SW_MX4 ? (MT == 4 ? 1 : 2) : (MT == 4 ? 2 : 4)>(a, sh, e, lane, wave);
}

template <int MT>
struct MoeDownShared {
  float own[kMoeWaves][16 * MT][16];
  uint32_t mask[kMoeExperts][2];     // tokens of an expert
  uint16_t active[kMoeExperts], place[kMoeExperts];
  uint16_t start[kMoeExperts + 1];
  uint32_t rows[16 * MT * kMoeTopK];   // token << 16 | pair, by expert
  int32_t expert[16 * MT * kMoeTopK];
  float prob[16 * MT * kMoeTopK];
  int n_active;
};

template <int WF, int DT, int MT>
__global__ __launch_bounds__(64 * kMoeWaves, MT < 2 ? 4 : 2) void moe_down_kernel(MoeArgs a) {
  __shared__ MoeDownShared<MT> sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kPairs = 16 * MT * kMoeTopK;
  constexpr int NT = 64 * kMoeWaves;
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
  float prob[(kPairs + NT - 1) / NT];
#pragma unroll
  for (int q = 0; q < (kPairs + NT - 1) / NT; ++q) {
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
  for (int q = 0; q < (kPairs + NT - 1) / NT; ++q) {
    const int i = tid + q * NT;
    if (i < pairs && sh.expert[i] >= 0) sh.prob[i] = prob[q];
  }
  __syncthreads();

  // This wave's share of the (expert, chunk) sequence, by groups of chunks of
  // one expert; the weights of the next group load while a group's are
  // multiplied, across experts too.
  constexpr int UC = WF == SW_MX4 ? (MT == 1 ? 2 : 1) : (MT == 4 ? 2 : 4);
  using S = Strip<WF, WF == SW_F16 ? SX_F16P : SX_BF16P, 1, MT, UC>;
  const int64_t h0 = (int64_t)blockIdx.x * 16;
  const int g = lane >> 4;
  const int cpe = (int)S::chunks(a.I), n = __builtin_amdgcn_readfirstlane(sh.n_active);
  const int64_t units = (int64_t)n * cpe;
  const int64_t u0 = units * wave / kMoeWaves, u1 = units * (wave + 1) / kMoeWaves;
  int64_t row = h0 + (lane & 15);
  if (row >= a.H) row = a.H - 1;
  const char* const w_row = a.w2 + row * a.w2_n;
  const uint8_t* const s_row = a.s2 + row * a.s2_n;
  auto weights = [&](int i) {
    const int64_t e = __builtin_amdgcn_readfirstlane(sh.active[i]);
    typename S::WPtr p;
    p.w[0] = w_row + e * a.w2_e;
    p.s[0] = s_row + e * a.s2_e;
    return p;
  };
  if (u0 < u1) {
    int i = (int)(u0 / cpe), c = (int)(u0 - (int64_t)i * cpe);
    int64_t left = u1 - u0;                                  // chunks from (i, c) on
    int end = left < cpe - c ? c + (int)left : cpe;          // of this wave, in expert i
    typename S::WPtr wp = weights(i);
    typename S::XPtr xp;
    xp.part = a.act_part;
    typename S::WBuf cur, nxt;
    typename S::XBuf x;
    uint32_t who[MT];
    int m = 0;
    f32x4 acc[1][MT];
    S::clear(acc);
    bool fresh = true;
    S::load_w(cur, wp, c, end, a.I, g);
    while (true) {
      if (fresh) {                                           // rows of the expert's tokens
        const int first = __builtin_amdgcn_readfirstlane(sh.start[i]);
        m = __builtin_amdgcn_readfirstlane(sh.start[i + 1]) - first;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const int p = 16 * t + (lane & 15);
          who[t] = sh.rows[first + (p < m ? p : m - 1)];
          xp.x[t] = a.act + (int64_t)(who[t] & 0xFFFFu) * a.act_row;
          xp.s[t] = nullptr;
        }
        fresh = false;
      }
      S::load_x(x, xp, c, end, a.I, g, m <= 16);
      // The next group: of this expert, or of the next one.
      const bool last_of_expert = c + UC >= end;
      const int64_t left_after = last_of_expert ? left - (end - c) : left - UC;
      const bool more = left_after > 0;
      const int i2 = last_of_expert ? i + 1 : i, c2 = last_of_expert ? 0 : c + UC;
      const int end2 = !last_of_expert ? end : (left_after < cpe ? (int)left_after : cpe);
      if (more) {
        if (last_of_expert) wp = weights(i2);
        S::load_w(nxt, wp, c2, end2, a.I, g);
      }
      S::mma(acc, cur, x, m <= 16);
      if (last_of_expert) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (16 * t + (lane & 15) < m) {
            const float p = sh.prob[who[t] & 0xFFFFu];
            float* q = &sh.own[wave][who[t] >> 16][4 * g];
#pragma unroll
            for (int r = 0; r < 4; ++r) q[r] += p * acc[0][t][r];
          }
        }
        S::clear(acc);
        fresh = true;
      }
      if (!more) break;
      cur = nxt;
      i = i2;
      c = c2;
      end = end2;
      left = left_after;
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * 4; i += NT) {
    const int t = i >> 2, g = i & 3;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kMoeWaves; ++w)
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
