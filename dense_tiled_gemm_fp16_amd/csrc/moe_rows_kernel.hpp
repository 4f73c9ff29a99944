// Tokens sorted by expert, and rows moved there and back (gfx950).
//
// A pair is a token t and one of its top_k choices j, number t top_k + j.  Sorted
// by expert and, within one, by number, pair number p has slot s: slots[p] = s,
// rows[s] = p.  Pairs whose expert is outside 0 .. E - 1 have no slot (-1), and
// the rows behind the last expert's are -1.
//
//   sort     a counting sort: a first kernel counts the experts of each chunk of
//            pairs; in the second a workgroup adds up the counts ahead of its
//            chunk, ranks the chunk's pairs (64 at a time: lanes of equal experts
//            find each other by one ballot per bit of the number) and writes both
//            tables.  A single chunk needs the second kernel only.  All sums are
//            of whole numbers, so the order of the LDS atomics among them is of
//            no consequence.
//   gather   a token's row is read once and written to its slots.
//   combine  a token's rows are read and added, in the order of its choices.
//   combine_backward  a token's gradient is read once; per choice the weighted
//            copy is written and the product with the expert's row summed up.
// The last three move rows of up to some ten KB with a few operations per
// element: memory bounds them.  Lanes take 16 bytes each, so that loads and
// stores are whole lines.  16384 tokens, top 8 of 64, 7168 bfloat16: sort 15 us,
// gather 360 to 425 (5.0 to 5.9 TB/s by where its rows lie, nearly all of it writes of
// rows in no order; in their order, reading x in no order, 520), combine 358 to 406,
// its gradients 730 to 780.  A token's slots are loaded one after another, in
// gather each behind the store ahead of it, which counts with few tokens: 48 of them in
// a graph 4.0, 4.5 and 3.9, the gradients 11.
#pragma once

#include "norm_kernel.hpp"

namespace gemmf16 {

constexpr int kSortExperts = 1024, kSortThreads = 512, kSortWaves = kSortThreads / 64;

struct SortArgs {
  const void* ids;
  int64_t ld;              // from token to token
  int32_t top_k, wide;     // wide: 64-bit ids
  int32_t E, bits;         // bits of a number below E
  int64_t P;               // pairs
  int64_t chunk, chunks;   // pairs of a chunk, a multiple of kSortThreads
  int32_t* counts;         // [chunks][E]; unused with one chunk
  int64_t* offsets;        // [E + 1]
  int64_t* rows;           // [P]
  int64_t* slots;          // [P]
};

// Expert of pair p, -1 if none.
__device__ __forceinline__ int pair_expert(const SortArgs& a, int64_t p) {
  if (p >= a.P) return -1;
  const int64_t t = p / a.top_k, at = t * a.ld + (p - t * a.top_k);
  const int64_t e = a.wide ? gload<int64_t>((const int64_t*)a.ids + at) : (int64_t)gload<int32_t>((const int32_t*)a.ids + at);
  return e >= 0 && e < a.E ? (int)e : -1;
}

__global__ __launch_bounds__(kSortThreads) void moe_count_kernel(SortArgs a) {
  __shared__ int count[kSortExperts];
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int64_t p0 = (int64_t)blockIdx.x * a.chunk;
  for (int64_t i = threadIdx.x; i < a.chunk; i += kSortThreads) {
    const int e = pair_expert(a, p0 + i);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = count[e];
}

__global__ __launch_bounds__(kSortThreads) void moe_place_kernel(SortArgs a) {
  __shared__ int hist[kSortWaves][kSortExperts];
  __shared__ int64_t total[kSortExperts], ahead[kSortExperts];   // of all chunks; of those before this one
  __shared__ int64_t scan[kSortThreads];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t c = blockIdx.x, sub = a.chunk / kSortWaves;      // pairs of a wave
  const int64_t p0 = c * a.chunk + wave * sub;
  for (int e = tid; e < a.E; e += kSortThreads) {
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) hist[i][e] = 0;
    total[e] = ahead[e] = 0;
  }
  __syncthreads();
  for (int64_t i = lane; i < sub; i += 64) {
    const int e = pair_expert(a, p0 + i);
    if (e >= 0) atomicAdd(&hist[wave][e], 1);
  }
  if (a.chunks > 1) {
    // Threads share out the chunks of each expert.
    const int group = a.E < kSortThreads ? kSortThreads / a.E : 1;   // threads of an expert
    for (int i = tid; i < a.E * group; i += kSortThreads) {
      const int e = i % a.E;
      int64_t all = 0, before = 0;
      for (int64_t q = i / a.E; q < a.chunks; q += group) {
        const int n = a.counts[q * a.E + e];
        all += n;
        before += q < c ? n : 0;
      }
      atomicAdd((unsigned long long*)&total[e], (unsigned long long)all);
      atomicAdd((unsigned long long*)&ahead[e], (unsigned long long)before);
    }
  }
  __syncthreads();
  if (a.chunks == 1) {
    for (int e = tid; e < a.E; e += kSortThreads) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kSortWaves; ++i) n += hist[i][e];
      total[e] = n;
    }
    __syncthreads();
  }
  // Exclusive sums over the experts: each thread a contiguous run of them.
  const int run = (a.E + kSortThreads - 1) / kSortThreads;
  const int e0 = tid * run < a.E ? tid * run : a.E, e1 = e0 + run < a.E ? e0 + run : a.E;
  int64_t sum = 0;
  for (int e = e0; e < e1; ++e) sum += total[e];
  scan[tid] = sum;
  __syncthreads();
  for (int d = 1; d < kSortThreads; d <<= 1) {
    const int64_t v = tid >= d ? scan[tid - d] : 0;
    __syncthreads();
    scan[tid] += v;
    __syncthreads();
  }
  int64_t at = tid > 0 ? scan[tid - 1] : 0;
  const int64_t placed = scan[kSortThreads - 1];
  for (int e = e0; e < e1; ++e) {
    if (c == 0) a.offsets[e] = at;
    ahead[e] += at;                       // the chunk's first slot of this expert
    at += total[e];
  }
  if (c == 0 && tid == 0) a.offsets[a.E] = placed;
  __syncthreads();
  for (int e = tid; e < a.E; e += kSortThreads) {   // each wave's first slot, from the chunk's
    int n = 0;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) {
      const int h = hist[i][e];
      hist[i][e] = n;
      n += h;
    }
  }
  __syncthreads();
  volatile int* mine = hist[wave];
  for (int64_t i = 0; i < sub; i += 64) {
    const int64_t p = p0 + i + lane;
    const int e = pair_expert(a, p);
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < a.bits; ++b) {
      const bool bit = (e >> b) & 1;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    int64_t slot = -1;
    if (e >= 0) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int before = mine[e];
      slot = ahead[e] + before + rank;
      // The lanes of an expert read before its last one writes: one wave, in
      // the order of the program.
      __builtin_amdgcn_wave_barrier();
      if ((same >> lane) == 1) mine[e] = before + rank + 1;
    }
    __builtin_amdgcn_wave_barrier();
    if (p < a.P) {
      a.slots[p] = slot;
      if (slot >= 0) a.rows[slot] = p;
    }
  }
  for (int64_t s = placed + c * kSortThreads + tid; s < a.P; s += a.chunks * kSortThreads) a.rows[s] = -1;
}

struct RowsArgs {
  const void* in;          // gather: tokens' rows; else the sorted rows
  int64_t ldi;             // bytes from row to row (also of the others)
  const void* dy;          // backward: tokens' gradients
  int64_t ldy;
  void* out;
  int64_t ldo;
  const int64_t* slots;    // [T][top_k]
  int64_t ld_slots;        // elements from token to token
  const int64_t* placed;   // gather and backward: rows of the experts (a device number)
  const void* weights;     // or null
  int64_t ldw;             // elements
  void* dweights;
  int64_t lddw;
  int64_t T, P, H;         // H: gather: bytes of a row; else elements
  int32_t top_k, w32, parts;
};

__device__ __forceinline__ int64_t slot_of(const RowsArgs& a, int64_t t, int j) {
  const int64_t s = a.slots[t * a.ld_slots + j];
  return s >= 0 && s < a.P ? s : -1;
}

// n (<= 16) bytes.
template <bool ONCE>
__device__ __forceinline__ void store_bytes(char* p, u32x4 v, int64_t n) {
  if (n >= 16) {
    gstore_once<ONCE>(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 15; ++i)
    if (i < n) gstore<uint8_t>((uint8_t*)p + i, (uint8_t)(v[i / 4] >> (8 * (i % 4))));
}

// Rows behind the experts' are zeros: workgroup t clears the top_k rows from
// number placed + t top_k.
template <int NT>
__device__ __forceinline__ void clear_rest(const RowsArgs& a, int64_t t, int64_t bytes, int64_t c0, int64_t c1) {
  int64_t n = *a.placed;
  n = n < 0 ? 0 : n < a.P ? n : a.P;     // a caller's offsets may hold anything
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t r = n + t * a.top_k + j;
    if (r >= a.P) return;
    for (int64_t c = c0 + threadIdx.x; c < c1; c += NT)
      store_bytes<false>((char*)a.out + r * a.ldo + 16 * c, zero4(), bytes - 16 * c);
  }
}

// Workgroups of 128 threads: parts of a token's row, its parts one after another,
// 16 bytes a lane.
constexpr int kRowThreads = 128;

template <bool ONCE>
__global__ __launch_bounds__(kRowThreads) void moe_gather_kernel(RowsArgs a) {
  const int64_t t = blockIdx.x / a.parts, chunks = (a.H + 15) / 16;
  const int64_t c0 = (int64_t)(blockIdx.x % a.parts) * kRowThreads, c = c0 + threadIdx.x;
  if (c < chunks) {
    const u32x4 v = load_bytes((const char*)a.in + t * a.ldi, 16 * c, a.H - 16 * c);
    for (int j = 0; j < a.top_k; ++j) {
      const int64_t s = slot_of(a, t, j);
      if (s >= 0) store_bytes<ONCE>((char*)a.out + s * a.ldo + 16 * c, v, a.H - 16 * c);
    }
  }
  clear_rest<kRowThreads>(a, t, a.H, c0, c0 + kRowThreads < chunks ? c0 + kRowThreads : chunks);
}

// Weight of choice j of token t, 1 without weights.
template <int FMT>
__device__ __forceinline__ float weight_of(const RowsArgs& a, int64_t t, int j) {
  if (!a.weights) return 1.0f;
  const int64_t at = t * a.ldw + j;
  if (a.w32) return ((const float*)a.weights)[at];
  return mx_in<FMT>(((const typename MxElem<FMT>::type*)a.weights)[at]);
}

template <int FMT, bool ONCE>
__device__ __forceinline__ void store_oct(char* row, int64_t k, const float (&f)[8], int64_t n) {
  if constexpr (FMT == MX_F32) {
    float* p = (float*)row + k;
    if (n >= 8) {
      gstore_once<ONCE>(p, f32x4{f[0], f[1], f[2], f[3]});
      gstore_once<ONCE>(p + 4, f32x4{f[4], f[5], f[6], f[7]});
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) gstore<float>(p + i, f[i]);
    }
  } else {
    store8_part<ONCE>((uint16_t*)row + k, pack8<FMT>(f), n);
  }
}

constexpr int kRowsAhead = 8;   // rows in flight, behind their slots

// An octet per lane, workgroups as above.
template <int FMT, bool ONCE>
__global__ __launch_bounds__(kRowThreads) void moe_combine_kernel(RowsArgs a) {
  const int64_t t = blockIdx.x / a.parts, k = 8 * ((int64_t)(blockIdx.x % a.parts) * kRowThreads + threadIdx.x);
  if (k >= a.H) return;
  float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < a.top_k; j0 += kRowsAhead) {
    Oct<FMT> v[kRowsAhead];
    int64_t s[kRowsAhead];
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      s[i] = j0 + i < a.top_k ? slot_of(a, t, j0 + i) : -1;
      v[i].template load<ONCE>((const char*)a.in + (s[i] < 0 ? 0 : s[i]) * a.ldi, k, s[i] < 0 ? 0 : a.H - k);
    }
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      // an absent row takes no part, whatever its weight
      const float w = s[i] >= 0 ? weight_of<FMT>(a, t, j0 + i) : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(w, v[i].get(e), sum[e]);
    }
  }
  store_oct<FMT, false>((char*)a.out + t * a.ldo, k, sum, a.H - k);
}

// Workgroup: a token.  Choices eight at a time; the token's gradient is read
// again for each further eight.
template <int FMT, bool ONCE>
__global__ __launch_bounds__(256) void moe_combine_back_kernel(RowsArgs a) {
  __shared__ float part[4][kRowsAhead];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j0 = 0; j0 < a.top_k; j0 += kRowsAhead) {
    int64_t s[kRowsAhead];
    float w[kRowsAhead], dot[kRowsAhead];
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      s[i] = j0 + i < a.top_k ? slot_of(a, t, j0 + i) : -1;
      w[i] = s[i] < 0 ? 0.0f : weight_of<FMT>(a, t, j0 + i);
      dot[i] = 0.0f;
    }
    for (int64_t k = 8 * (int64_t)threadIdx.x; k < a.H; k += 8 * 256) {
      Oct<FMT> g, v[kRowsAhead];
      g.load((const char*)a.dy + t * a.ldy, k, a.H - k);
#pragma unroll
      for (int i = 0; i < kRowsAhead; ++i)
        v[i].template load<ONCE>((const char*)a.in + (s[i] < 0 ? 0 : s[i]) * a.ldi, k, s[i] < 0 ? 0 : a.H - k);
#pragma unroll
      for (int i = 0; i < kRowsAhead; ++i) {
        if (s[i] < 0) continue;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] = w[i] * g.get(e);
          dot[i] = __builtin_fmaf(g.get(e), v[i].get(e), dot[i]);
        }
        store_oct<FMT, ONCE>((char*)a.out + s[i] * a.ldo, k, f, a.H - k);
      }
    }
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      const float d = wave_sum(dot[i]);
      if (lane == 0) part[wave][i] = d;
    }
    __syncthreads();
    if (threadIdx.x < kRowsAhead && j0 + (int)threadIdx.x < a.top_k) {
      const int i = threadIdx.x;
      const float d = part[0][i] + part[1][i] + part[2][i] + part[3][i];   // zero without a slot
      const int64_t at = t * a.lddw + j0 + i;
      if (a.w32)
        ((float*)a.dweights)[at] = d;
      else if constexpr (FMT != MX_F32)
        ((uint16_t*)a.dweights)[at] = cvt_out<FMT == MX_F16 ? DT_F16 : DT_BF16>(d);
    }
    __syncthreads();
  }
  const int64_t bytes = a.H * Oct<FMT>::ES;
  clear_rest<256>(a, t, bytes, 0, (bytes + 15) / 16);
}

}  // namespace gemmf16
