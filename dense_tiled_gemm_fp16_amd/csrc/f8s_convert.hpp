// Quantisation to FP8 with a float32 scale for each block of 128 (gfx950).
//
// With m the largest magnitude of a block and L the format's largest value the
// scale is max(m, L 2^-126) / L, and an element x becomes x L / max(m, ..)
// rounded to nearest even.  The quotient is not x over the rounded scale: 16-bit
// elements often lie exactly midway between two 8-bit values, and the scale's
// own rounding would decide all those ties of a block the same way.
//
// In float32 the quotient of a 16-bit x is correctly rounded: with m = f 2^e,
// X = x (L 2^-e) is exact (11 + 3 bits), t = X (1 / f) is off by two units at
// most, and one residual X - t f by fused multiply-add brings it home.  A
// quotient that is a tie between two 8-bit values is therefore met exactly, and
// no other one of 16-bit numbers is near enough to a tie to round onto it.
//
// Both kernels are one pass over memory (2 or 4 bytes read, 1 + 1/32 written),
// which bounds them:
//   rows   blocks of one row, k contiguous: a lane takes 8 consecutive elements
//          (one 16-byte load of a 16-bit type), 16 neighbouring lanes a block,
//          whose maximum goes round them by four lane exchanges in registers.
//          A wave has four such loads in flight; short rows share them.  32768 x
//          7168 bfloat16 110 us (6.4 TB/s), 8192 x 7168 35.
//   tiles  blocks of 128 rows x 128 elements, or of one row where k is strided: a
//          workgroup takes 128 x 128 elements, a thread 8 x 8 of them, loaded
//          along the contiguous axis.  Rows of k-strided input leave through LDS
//          so that stores are whole lines.  8192 x 7168 bfloat16 along the columns
//          44 us, in square blocks 37; as wide floats from the load on, with twice
//          the registers and lane exchanges, 54 and 41.
#pragma once

#include "f8_kernel.hpp"
#include "mx4_convert.hpp"

namespace gemmf16 {

constexpr int kF8Block = 128;

template <int F8>
__device__ __forceinline__ uint32_t f8_largest_bits() {
  return F8 == F8_E4M3 ? 0x43E00000u : 0x47600000u;   // 448, 57344
}

struct F8Scale {
  float scale, up, f, rf;   // X = x up, quotient X / f
  bool bad;                 // an infinity or a NaN in the block
};

// From the bits of the block's largest magnitude.
template <int F8>
__device__ __forceinline__ F8Scale f8_scale(uint32_t m) {
  const uint32_t lb = f8_largest_bits<F8>();
  const float L = __builtin_bit_cast(float, lb);
  F8Scale s;
  s.bad = m >= 0x7F800000u;
  const uint32_t least = lb - (126u << 23);                // L 2^-126
  if (m < least) m = least;
  // m / L: the quotient by L's reciprocal, with its residual's correction.
  const float v = __builtin_bit_cast(float, m), rl = 1.0f / L;               // rl: a constant
  const float q = v * rl;
  s.scale = s.bad ? __builtin_nanf("") : __builtin_fmaf(__builtin_fmaf(-q, L, v), rl, q);
  s.f = __builtin_bit_cast(float, (m & 0x007FFFFFu) | 0x3F800000u);
  s.up = __builtin_bit_cast(float, lb - (m & 0x7F800000u) + (127u << 23));   // L 2^-e
  const float r = __builtin_amdgcn_rcpf(s.f);                                // one Newton step
  s.rf = __builtin_fmaf(__builtin_fmaf(-s.f, r, 1.0f), r, r);
  return s;
}

// Rounded once for a 16-bit x; else twice, with x up itself.
__device__ __forceinline__ float f8_quotient(float x, const F8Scale& s) {
  const float X = x * s.up;
  const float t = X * s.rf;
  return __builtin_fmaf(__builtin_fmaf(-t, s.f, X), s.rf, t);
}

// 8 floats -> 8 codes, the first in the lowest byte; zeros for a bad block.
template <int F8>
__device__ __forceinline__ u32x2 f8_codes(const float (&x)[8], const F8Scale& s) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = f8_quotient(x[i], s);
  int d[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (F8 == F8_E4M3) {
      d[h] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], d[h], false);
      d[h] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], d[h], true);
    } else {
      d[h] = __builtin_amdgcn_cvt_pk_bf8_f32(q[4 * h], q[4 * h + 1], d[h], false);
      d[h] = __builtin_amdgcn_cvt_pk_bf8_f32(q[4 * h + 2], q[4 * h + 3], d[h], true);
    }
  }
  return s.bad ? u32x2{0u, 0u} : u32x2{(uint32_t)d[0], (uint32_t)d[1]};
}

// Largest of 16 neighbouring lanes' values, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  auto take = [&](uint32_t o) { v = o > v ? o : v; };
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));    // lane ^ 1
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));    // lane ^ 2
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));   // mirrored in 8
  take((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));   // mirrored in 16
  return v;
}

__device__ __forceinline__ uint32_t magnitude(float f) { return __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu; }

// The first n (<= 8) of 8 codes.
template <bool ONCE = false>
__device__ __forceinline__ void store_codes(uint8_t* p, u32x2 v, int64_t n) {
  if (n >= 8) {
    gstore_once<ONCE>(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) gstore<uint8_t>(p + i, (uint8_t)(v[i / 4] >> (8 * (i % 4))));
}

struct F8QuantArgs {
  const void* x;
  int64_t s_r, s_k;        // element strides
  int64_t R, K;
  uint8_t* data;
  int64_t ldd;
  float* scales;
  int64_t ss_r, ss_k;      // from scale row to scale row, from block to block
  int64_t segs;            // rows: wave items per row; tiles: blocks along K
  Short few;
};

// The larger of two magnitudes, of both halves in 16-bit formats (whose bits order
// them as float32's do).
template <int FMT>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  if constexpr (FMT == MX_F32) return a > b ? a : b;
  using half2 = uint16_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(half2, a), __builtin_bit_cast(half2, b)));
}
// Largest magnitudes of N lines of 8 elements, of each element on its own.
template <int FMT, int N>
__device__ __forceinline__ Oct<FMT> largest_of(const Oct<FMT> (&v)[N]) {
  Oct<FMT> m;
#pragma unroll
  for (int h = 0; h < Oct<FMT>::ES / 2; ++h)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t x = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) x = larger<FMT>(x, v[i].v[h][w] & (FMT == MX_F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu));
      m.v[h][w] = x;
    }
  return m;
}

// Bits of the largest of 8 magnitudes, as a float32's.
template <int FMT>
__device__ __forceinline__ uint32_t largest_bits(const Oct<FMT>& m) {
  Oct<FMT> one = m;
  uint32_t x = 0;
#pragma unroll
  for (int h = 0; h < Oct<FMT>::ES / 2; ++h)
#pragma unroll
    for (int w = 0; w < 4; ++w) x = larger<FMT>(x, m.v[h][w]);
  one.v[0][0] = x;
  if constexpr (FMT == MX_F32) return x;
  const uint32_t a = magnitude(one.get(0)), b = magnitude(one.get(1));
  return a > b ? a : b;
}

// Rows with unit k stride; wave items as in quantize_rows_kernel, with 16 octets
// a block.
template <int FMT, int F8, bool SHORT, bool ONCE>
__global__ __launch_bounds__(256) void f8_rows_kernel(F8QuantArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t w = wave_item();
  const int64_t octs = 16 * ((a.K + kF8Block - 1) / kF8Block);
  Oct<FMT> v[kQuantU];
#pragma unroll
  for (int u = 0; u < kQuantU; ++u) {
    const Place p = place<SHORT>(w, u, lane, a.R, octs, a.segs, a.few);
    v[u].template load<ONCE>((const char*)a.x + p.row * a.s_r * Oct<FMT>::ES, 8 * p.o, p.ok ? a.K - 8 * p.o : 0);
  }
#pragma unroll
  for (int u = 0; u < kQuantU; ++u) {
    const Place p = place<SHORT>(w, u, lane, a.R, octs, a.segs, a.few);
    const Oct<FMT> line[1] = {v[u]};
    const F8Scale s = f8_scale<F8>(max16(largest_bits(largest_of(line))));
    if (p.ok) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = v[u].get(i);
      store_codes<ONCE>(a.data + p.row * a.ldd + 8 * p.o, f8_codes<F8>(f, s), a.K - 8 * p.o);
      if ((p.o & 15) == 0) gstore<float>(a.scales + p.row * a.ss_r + (p.o >> 4) * a.ss_k, s.scale);
    }
  }
}

// 8 elements `step` apart in memory, `valid` of them.
template <int FMT, bool ONCE>
__device__ __forceinline__ void load8_strided(Oct<FMT>& v, const void* x, int64_t at, int64_t step, int64_t valid) {
  if (step == 1) {
    v.template load<ONCE>(x, at, valid);
    return;
  }
  const char* p = (const char*)x + at * Oct<FMT>::ES;
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    typename MxElem<FMT>::type e = 0;
    if (i < valid) e = gload<typename MxElem<FMT>::type>(p + i * step * Oct<FMT>::ES);
    h[i] = e;
  }
  if constexpr (FMT == MX_F32) {
    v.v[0] = u32x4{h[0], h[1], h[2], h[3]};
    v.v[1] = u32x4{h[4], h[5], h[6], h[7]};
  } else {
    v.v[0] = u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
  }
}

// One 128 x 128 tile.  ALONG_K: a thread's 8 loads are 8 rows of 8 consecutive k
// (threads of a row: 16 neighbouring lanes); else 8 k of 8 consecutive rows.
template <int FMT, int F8, bool SQUARE, bool ALONG_K, bool ONCE>
__global__ __launch_bounds__(256) void f8_tiles_kernel(F8QuantArgs a) {
  static_assert(SQUARE || !ALONG_K, "rows with unit k stride have their own kernel");
  __shared__ __attribute__((aligned(16))) uint32_t part[4 * kF8Block];
  __shared__ __attribute__((aligned(16))) char turn[SQUARE && ALONG_K ? 16 : kF8Block * 128];
  const int tid = threadIdx.x, hi = tid >> 4, lo = tid & 15, lane = tid & 63, wave = tid >> 6;
  const int64_t tile = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t br = tile / a.segs, bk = tile - br * a.segs;
  if (br * kF8Block >= a.R) return;
  // The thread's 8 x 8 elements: rows r0 .., k from q0.
  const int rl = 8 * (ALONG_K ? hi : lo), kl = 8 * (ALONG_K ? lo : hi);
  const int64_t r0 = br * kF8Block + rl, q0 = bk * kF8Block + kl;
  const int64_t nr = a.R - r0, nk = a.K - q0;
  Oct<FMT> v[8];           // [line][element]: ALONG_K [row][k], else [k][row]
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t at = ALONG_K ? (r0 + i) * a.s_r + q0 * a.s_k : (q0 + i) * a.s_k + r0 * a.s_r;
    const bool ok = i < (ALONG_K ? nr : nk);
    load8_strided<FMT, ONCE>(v[i], a.x, at, ALONG_K ? a.s_k : a.s_r, ok ? (ALONG_K ? nk : nr) : 0);
  }
  Oct<FMT> most = largest_of(v);
  F8Scale s[SQUARE ? 1 : 8];
  if constexpr (SQUARE) {
    uint32_t m = max16(largest_bits(most));
    if (lo == 0) part[hi] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = part[i] > m ? part[i] : m;
    s[0] = f8_scale<F8>(m);
    if (tid == 0) a.scales[br * a.ss_r + bk * a.ss_k] = s[0].scale;
  } else {
    // Row rl + e: over this thread's 8 k, the wave's four groups of 16 lanes,
    // the four waves.
    constexpr int H = Oct<FMT>::ES / 2;
    u32x4* const rows = reinterpret_cast<u32x4*>(part);       // [wave][lo][H]
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t m = most.v[h][w];
        m = larger<FMT>(m, (uint32_t)__shfl_xor((int)m, 16));
        most.v[h][w] = larger<FMT>(m, (uint32_t)__shfl_xor((int)m, 32));
      }
      if (lane < 16) rows[(wave * 16 + lo) * H + h] = most.v[h];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < H; ++h) {
      u32x4 m = rows[lo * H + h];
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        const u32x4 o = rows[(i * 16 + lo) * H + h];
#pragma unroll
        for (int w = 0; w < 4; ++w) m[w] = larger<FMT>(m[w], o[w]);
      }
      most.v[h] = m;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = f8_scale<F8>(magnitude(most.get(e)));
    // its scale by the first k's thread
    if (hi == 0)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < nr) a.scales[(r0 + e) * a.ss_r + bk * a.ss_k] = s[e].scale;
  }
  if constexpr (ALONG_K) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nr) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[i].get(e);
        store_codes<ONCE>(a.data + (r0 + i) * a.ldd + q0, f8_codes<F8>(f, s[0]), nk);
      }
  } else {
    // Row e's 8 k into LDS (rows of 128 bytes, 8-byte chunk c of row r in slot
    // c ^ (r / 8) % 16: the 16 rows 8 apart that neighbouring lanes write fall on
    // distinct banks), back as whole rows.
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = v[i].get(e);
      *reinterpret_cast<u32x2*>(turn + (rl + e) * 128 + ((hi ^ lo) * 8)) = f8_codes<F8>(f, s[SQUARE ? 0 : e]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 16 * i + hi;
      const int64_t row = br * kF8Block + r, k = bk * kF8Block + 8 * lo;
      const u32x2 v = *reinterpret_cast<const u32x2*>(turn + r * 128 + ((lo ^ (r >> 3)) * 8));
      if (row < a.R) store_codes<ONCE>(a.data + row * a.ldd + k, v, a.K - k);
    }
  }
}

}  // namespace gemmf16
