// A mixture-of-experts layer for a few tokens in two kernels (gfx950), three
// where there are few columns.
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
//             bfloat16 parts per value, into row (token, slot).  The waves of a
//             workgroup are kMoeWaves / parts neighbouring strips times the
//             parts: as few parts as still fill the device, so that a wave
//             streams long rows and the workgroup's waves meet A in L1.  With
//             fewer (token, slot) pairs than experts, a workgroup is tied to a
//             pair instead, and only the first pair of an expert goes on.  The
//             workgroups of the first strips also write the pair's expert and
//             its softmax weight.
//   moe_down  workgroup -> 16 NS columns of Y, all experts: the waves share the
//             (expert, chunk of I) sequence evenly, loads running ahead across
//             experts, each adds p * (sums) into its own [T, 16 NS] accumulators
//             in LDS at every expert's end, and the waves' accumulators are
//             added in order.  So the weighted sum over experts needs no
//             atomics and no further pass.  Where the columns give too few
//             workgroups, `splits` of them share the sequence of a strip, and
//             moe_sum adds their sums in order.
//
// Measured (us, medians of a kernel trace, H 7168, I 2048, top 8 of 64 experts;
// what the weights take at the 6.4 TB/s of plain reads in brackets): bfloat16, 1
// token 75 + 43 (73 + 37), 64 tokens 592 + 324 (587 + 294; binary16 592 + 397, see
// split_parts); MX4, 16 tokens 208 + 135 (139 + 69), where scale bytes fetched
// more than once, LDS and conversions take the rest, 64 tokens 285 + 215 (156 +
// 78).  In a graph the layer takes 118, 879, 309 and 464.
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
  float* sums;                 // [splits][T][sums_row] of moe_down, where it is split
  int64_t sums_row;
  int64_t H, I;
  int32_t T, E, k, fmt_l, by_pair, renormalize;
  int32_t parts;               // of H, in moe_up: 1, 2, 4 or 8
  int32_t splits;              // of moe_down: workgroups per strip of columns
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
  if (a.fmt_l == 2) return gload<float>((const float*)a.logits + i);
  const uint16_t h = gload<uint16_t>((const uint16_t*)a.logits + i);
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

// silu(g) u as two bfloat16 parts, what the down product takes: fp32 does not
// enter the 16-bit matrix instructions, and two parts keep 2^-16 of a value (the
// output keeps 2^-8 or 2^-11) over fp32's whole range.  Beside binary16 weights
// too, which the down product then splits (4 tokens, top 2 of 16, H 2048, I 768,
// in a graph: the layer 27.1 us, with binary16 parts 25.0; 64 tokens, top 8 of 64,
// H 7168, I 2048: 926 to 945 and 878): binary16 parts keep more of a value near 1, but their least
// step is 2^-24 and they end at 65504, while silu(g) u may lie below and above.
__device__ __forceinline__ void split_parts(float v, uint16_t& hi, uint16_t& lo) {
  hi = cvt_out<DT_BF16>(v);
  const float r = v - cvt_in<DT_BF16>(hi);
  lo = cvt_out<DT_BF16>(r == r && fabsf(r) <= fabsf(v) ? r : 0.0f);   // nothing beside an infinity or a NaN
}

// What a wave of moe_up takes: NI strips of 16 rows of I (gate and up: 2 NI
// strips of W1), UC chunks at a time.
template <int WF, int DT, int MT, int NI_, int UC, bool ONCE>
struct MoeUp {
  static constexpr int NI = NI_;
  using S = Strip<WF, DT == DT_F16 ? SX_F16 : SX_BF16, 2 * NI, MT, UC, 1, false,
                  ONCE>;   // few experts get more than 16 tokens
  static constexpr int TILES = 2 * NI * MT;

  struct Shared {
    union {
      char wave[kMoeWaves][S::LDS];
      f32x4 part[kMoeWaves * TILES * 64];
      uint32_t key[kMoeExperts];
    };
    int rank[kMoeTokens];     // slot of the expert in the token's choice, -1 not chosen
    int list[kMoeTokens];     // the expert's tokens
    int count, found;
  };

  static __device__ __forceinline__ void run(const MoeArgs& a, Shared& sh, int e, int lane, int wave) {
    const int m = __builtin_amdgcn_readfirstlane(sh.count), tiles = (m + 15) / 16;
    const int strips = kMoeWaves / a.parts;      // of this workgroup
    const int strip = wave / a.parts, part = wave - strip * a.parts;
    const int64_t i0 = ((int64_t)blockIdx.x * strips + strip) * (16 * NI);
    f32x4 acc[2 * NI][MT];
    S::clear(acc);
    if (i0 < a.I) {
      const typename S::WPtr w{a.w1 + e * a.w1_e + i0 * a.w1_n, a.s1 + e * a.s1_e + i0 * a.s1_n};
      typename S::WOff wo;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NI; ++n) {
#pragma unroll
          for (int j = 0; j < UC; ++j) {
            int64_t row = 16 * n + S::w_row(j, lane);
            if (row >= a.I - i0) row = a.I - i0 - 1;
            wo.w[h * NI + n][j] = (uint32_t)((h * a.I + row) * a.w1_n) + 16 * (lane % S::WP);
          }
          int64_t srow = 16 * n + (lane < 16 ? lane : 0);
          if (srow >= a.I - i0) srow = a.I - i0 - 1;
          wo.s[h * NI + n] = (uint32_t)((h * a.I + srow) * a.s1_n);
        }
      auto rows = [&](int p, int) {
        typename S::XPtr x;
        x.x = a.x;
        x.xo = (uint32_t)(sh.list[p < m ? p : m - 1] * a.ldx);
        x.s = nullptr;
        x.so = 0;
        return x;
      };
      S::run(acc, sh.wave[wave], w, wo, rows, 0, part, a.parts, a.H, m, lane);
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2 * NI; ++h)
#pragma unroll
      for (int t = 0; t < MT; ++t) sh.part[(wave * TILES + h * MT + t) * 64 + lane] = acc[h][t];
    __syncthreads();
    for (int j = wave; j < strips * NI * tiles; j += kMoeWaves) {
      const int t = j % tiles, n = j / tiles % NI, s = j / (tiles * NI);
      const f32x4* base = sh.part + s * a.parts * TILES * 64 + (n * MT + t) * 64;
      const int p = 16 * t + (lane & 15);
      const int64_t i = (((int64_t)blockIdx.x * strips + s) * NI + n) * 16 + 4 * (lane >> 4);
      if (p < m && i < a.I) {       // rows hold a multiple of 8 values: all four fit
        const f32x4 gate = sum_waves(base, TILES * 64, a.parts, lane);
        const f32x4 up = sum_waves(base + NI * MT * 64, TILES * 64, a.parts, lane);
        const int token = sh.list[p];
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          split_parts(gate[r] / (1.0f + expf(-gate[r])) * up[r], hi[r], lo[r]);
        char* q = a.act + (token * a.k + sh.rank[token]) * a.act_row + 2 * i;
        gstore(q, u32x2{hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16});
        gstore(q + a.act_part, u32x2{lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16});
      }
    }
  }
};

// Grid (groups of strips of rows of I, experts or pairs).  DT: format of X; MT:
// tiles of 16 tokens that T needs.
template <int WF, int DT, int MT, int NI, int UC, int WPS, bool ONCE>
__global__ __launch_bounds__(64 * kMoeWaves, WPS) void moe_up_kernel(MoeArgs a) {
  using U = MoeUp<WF, DT, MT, NI, UC, ONCE>;
  __shared__ typename U::Shared sh;
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
  U::run(a, sh, e, lane, wave);
}

// Four columns of a row of Y.
template <int DT>
__device__ __forceinline__ void store_y(const MoeArgs& a, int t, int64_t h, const f32x4& s) {
  uint16_t* y = a.y + t * a.ldy + h;
  uint16_t o[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] = cvt_out<DT>(s[r]);
  if (h + 4 <= a.H) {
    gstore(y, u32x2{o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16});
  } else {
    for (int r = 0; r < 4 && h + r < a.H; ++r) gstore<uint16_t>(y + r, o[r]);
  }
}

// What a workgroup of moe_down takes: NS strips of 16 columns of Y, 16 MT
// tokens.  FEW: an expert seldom has more than four tokens (see Strip).
template <int WF, int MT, int NS_, int UC, bool FEW, bool ONCE>
struct MoeDown {
  static constexpr int NS = NS_, NW = kMoeWaves;
  using S = Strip<WF, SX_BF16P, NS, FEW ? 2 * MT : MT, UC, 1, FEW, ONCE>;
  static constexpr int kPairs = 16 * MT * kMoeTopK;

  struct Shared {
    char wave[NW][S::LDS];
    float own[NW][16 * MT][16 * NS];
    uint32_t mask[kMoeExperts][2];     // tokens of an expert
    uint16_t active[kMoeExperts], place[kMoeExperts];
    uint16_t start[kMoeExperts + 1];
    uint32_t rows[kPairs];             // token << 16 | pair, by expert
    int32_t expert[kPairs];
    float prob[kPairs];
    int n_active;
  };
};

template <int WF, int DT, int MT, int NS, int UC, int WPS, bool FEW, bool ONCE>
__global__ __launch_bounds__(64 * kMoeWaves, WPS) void moe_down_kernel(MoeArgs a) {
  using D = MoeDown<WF, MT, NS, UC, FEW, ONCE>;
  using S = typename D::S;
  constexpr int kPairs = D::kPairs;
  __shared__ typename D::Shared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int NW = D::NW, NT = 64 * NW;
  const int pairs = a.T * a.k;
  for (int i = tid; i < a.E; i += NT) sh.mask[i][0] = sh.mask[i][1] = 0;
  for (int i = tid; i < pairs; i += NT) {
    sh.expert[i] = a.tab_e[i];
    sh.prob[i] = a.tab_p[i];
  }
  for (int i = lane; i < a.T * (16 * NS); i += 64) sh.own[wave][i / (16 * NS)][i % (16 * NS)] = 0.0f;
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

  // The whole groups of chunks of all experts, dealt to the waves of all
  // workgroups of the strip in turn (a row's neighbouring pieces are then read
  // at about the same time), loads running ahead across experts; then the
  // partial groups, if I has one.
  const int first_wave = blockIdx.y * NW + wave, waves = a.splits * NW;
  const int64_t h0 = (int64_t)blockIdx.x * (16 * NS);
  const int n = __builtin_amdgcn_readfirstlane(sh.n_active);
  struct Cursor {
    const MoeArgs* a;
    const typename D::Shared* sh;
    int64_t h0;
    int i, n, g, gpe, waves, first, m;     // group g of gpe of expert i of n
    __device__ __forceinline__ void at_expert() {
      while (g >= gpe && i < n) {
        g -= gpe;
        ++i;
      }
      if (i < n) {
        first = __builtin_amdgcn_readfirstlane(sh->start[i]);
        m = __builtin_amdgcn_readfirstlane(sh->start[i + 1]) - first;
      }
    }
    __device__ __forceinline__ bool more() const { return i < n; }
    __device__ __forceinline__ bool last() const { return g + waves >= gpe; }   // of the wave's, in an expert
    __device__ __forceinline__ void next() {
      g += waves;
      at_expert();
    }
    __device__ __forceinline__ int64_t c() const { return (int64_t)g * S::UC; }
    __device__ __forceinline__ typename S::WPtr w() const {
      const int64_t e = __builtin_amdgcn_readfirstlane(sh->active[i]);
      return {a->w2 + e * a->w2_e + h0 * a->w2_n, a->s2 + e * a->s2_e + h0 * a->s2_n};
    }
    __device__ __forceinline__ typename S::XPtr x(int p, int = 0) const {
      typename S::XPtr x;
      x.x = a->act;
      x.xo = (sh->rows[first + (p < m ? p : m - 1)] & 0xFFFFu) * (uint32_t)a->act_row;
      x.s = nullptr;
      x.so = 0;
      return x;
    }
    __device__ __forceinline__ int rows() const { return m; }
  };
  {
    char* const lds = sh.wave[wave];
    const typename S::WOff wo = S::offsets(a.H - h0, 16, a.w2_n, a.s2_n, lane);
    const int gpe = (int)S::groups(a.I);
    f32x4 acc[NS][S::MT];
    S::clear(acc);
    // p times an expert's sums into the wave's accumulators.
    auto add = [&](const Cursor& cc) {
#pragma unroll
      for (int t = 0; t < S::MT; ++t) {
        if constexpr (S::PACK) {
          if (S::TR * t >= cc.m) break;
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[s][t][r] += __shfl_xor(acc[s][t][r], S::TR);
        }
        const int p = S::TR * t + (lane & 15);
        if (p < cc.m && (lane & 15) < S::TR) {
          const uint32_t who = sh.rows[cc.first + p];
          const float prob = sh.prob[who & 0xFFFFu];
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            float* q = &sh.own[wave][who >> 16][16 * s + 4 * (lane >> 4)];
#pragma unroll
            for (int r = 0; r < 4; ++r) q[r] += prob * acc[s][t][r];
          }
        }
      }
      S::clear(acc);
    };
    if (gpe > 0) {
      Cursor cur{&a, &sh, h0, 0, n, first_wave, gpe, waves, 0, 0};
      cur.at_expert();
      S::stream(acc, lds, cur, wo, a.act_part, a.I, lane, [&](const Cursor& cc) {
        if (cc.last()) add(cc);
      });
    }
    if (S::rest(a.I))
      for (int i = first_wave; i < n; i += waves) {
        Cursor cur{&a, &sh, h0, i, n, 0, gpe + 1, waves, 0, 0};
        cur.at_expert();
        cur.g = gpe;
        S::finish(acc, lds, cur, wo, a.act_part, a.I, lane);
        add(cur);
      }
  }
  __syncthreads();
  // The waves' sums in order.
  for (int i = tid; i < a.T * (4 * NS); i += NT) {
    const int t = i / (4 * NS), g = i % (4 * NS);
    f32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] += sh.own[w][t][4 * g + r];
    if (a.splits == 1)
      store_y<DT>(a, t, h0 + 4 * g, s);
    else
      gstore(a.sums + ((int64_t)blockIdx.y * a.T + t) * a.sums_row + h0 + 4 * g, s);
  }
}

// The splits' sums in order: thread -> four columns of a token.
template <int DT>
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeArgs a) {
  const int t = blockIdx.y;
  const int64_t h = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (h >= a.H) return;
  f32x4 s{0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < a.splits; ++p) {
    const f32x4 v = gload<f32x4>(a.sums + ((int64_t)p * a.T + t) * a.sums_row + h);
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] += v[r];
  }
  store_y<DT>(a, t, h, s);
}

}  // namespace gemmf16
