// Quantisation to MX FP4 and back (gfx950).
//
// Both are one pass over memory: a few operations per element against 2 to 4
// bytes read and 17/32 written (or the reverse), so the memory rate bounds
// them and the kernels only have to keep wide loads in flight.
//
//   rows     k is the contiguous axis.  A lane takes 8 consecutive elements
//            (one 16-byte load of a 16-bit type), four neighbouring lanes a
//            block; the block's largest magnitude goes round the four with
//            two lane exchanges.  A wave has U such loads in flight; rows
//            of up to their 2048 elements share them.
//   columns  any other strides: a lane owns a row and walks the 32 elements of
//            a block, so that with rows contiguous a wave's loads cover 64
//            consecutive elements; no lane exchange is needed.  The codes go
//            through LDS to be stored in whole lines.
//
// Measured (us; TB/s read plus written; a copy reaches 4.7): 32768 x 7168 rows
// from bfloat16 and back 239 in a graph (5.0), in a kernel trace 113 to 129 (4.6 to
// 5.3) and 108 to 114 (5.2 to 5.5);
// fp32 201 (5.3) and 195 (5.5; two 16-byte stores per lane, 32 bytes apart,
// instead of side by side: 272); columns of bfloat16 131 (4.5; each lane storing
// its own 16 bytes: 176); 30000 x 333 padded rows 9.6 each (a wave per row: 16.8
// and 11.9).
//
// The scale's exponent is read off the magnitude's own bits: floor(log2 m) is
// the exponent field of a normal float, and a subnormal m (only from fp32 or
// bfloat16) clamps to the least scale anyway.  Division by the scale is an
// exact multiplication by 2^(127 - byte), after which the packed convert
// rounds to nearest even and saturates at 6.
#pragma once

#include "mx4_common.hpp"

namespace gemmf16 {

enum MxFormat { MX_F16 = 0, MX_BF16 = 1, MX_F32 = 2 };

// Rows of at most kSlots octets: a wave item takes `rows` of them, slot i octet
// i % octs of row i / octs, the division by a 16-bit reciprocal (exact for
// i < 256: i times its error stays below 1 / 256).
constexpr int kQuantU = 4, kSlots = 64 * kQuantU;   // octets in flight: U per lane
struct Short {
  int32_t octs, rows, inv;
};

struct QuantArgs {
  const void* x;
  int64_t s_g, s_r, s_k;   // element strides
  int64_t G, R, K;
  uint8_t* data;           // [G R, 16 Kb]
  uint8_t* scales;         // [G R, Kb]
  int64_t Kb;              // blocks per row
  int64_t segs;            // rows: wave items per row; columns: workgroups per strip of 64 rows
  Short few;               // rows: several rows per wave item
};

template <int FMT>
struct MxElem {
  using type = uint16_t;
};
template <>
struct MxElem<MX_F32> {
  using type = uint32_t;
};

template <int FMT>
__device__ __forceinline__ float mx_in(typename MxElem<FMT>::type v) {
  if constexpr (FMT == MX_F32)
    return __builtin_bit_cast(float, v);
  else
    return cvt_in<FMT == MX_F16 ? DT_F16 : DT_BF16>(v);
}

// 8 consecutive elements as they lie, n of them valid (the rest zero).
template <int FMT>
struct Oct {
  static constexpr int ES = FMT == MX_F32 ? 4 : 2;
  u32x4 v[ES / 2];

  template <bool ONCE = false>
  __device__ __forceinline__ void load(const void* base, int64_t k, int64_t n) {
    const char* p = (const char*)base + k * ES;
    if (n >= 8) {
      v[0] = load16_once<ONCE>(p);
      if constexpr (FMT == MX_F32) v[1] = load16_once<ONCE>(p + 16);
      return;
    }
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      typename MxElem<FMT>::type e = 0;
      if (i < n) e = gload<typename MxElem<FMT>::type>(p + i * ES);
      h[i] = e;
    }
    if constexpr (FMT == MX_F32) {
      v[0] = u32x4{h[0], h[1], h[2], h[3]};
      v[1] = u32x4{h[4], h[5], h[6], h[7]};
    } else {
      v[0] = u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (FMT == MX_F32) {
      const uint32_t e = v[i / 4][i % 4];   // a copy: bit_cast of a vector's element reads element 0
      return __builtin_bit_cast(float, e);
    } else
      return mx_in<FMT>((uint16_t)(v[0][i / 2] >> (16 * (i & 1))));
  }
};

// Scale byte of a block whose largest magnitude has these bits (the sign
// cleared; an infinity or a NaN among the elements compares largest).
__device__ __forceinline__ uint32_t scale_of(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255 ? 255u : (e < 2 ? 0u : e - 2);
}
// 2^(127 - byte): exact, normal for every byte but 254 and 255, which
// scale_of does not give below an infinity.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return __builtin_bit_cast(float, (254u - byte) << 23);
}

// 8 floats over their scale -> 8 codes.
__device__ __forceinline__ uint32_t to_codes(const float* f, uint32_t byte) {
  if (byte == 255) return 0;
  const float r = inverse_scale(byte);
  uint32_t d = 0;
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, f[0] * r, f[1] * r, 1.0f, 0);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, f[2] * r, f[3] * r, 1.0f, 1);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, f[4] * r, f[5] * r, 1.0f, 2);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, f[6] * r, f[7] * r, 1.0f, 3);
  return d;
}

// The wave's number in a grid that may spill over into y.
__device__ __forceinline__ int64_t wave_item() {
  return ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// Where a lane's u-th octet of a wave item lies.
struct Place {
  int64_t row, o;
  bool ok;
};
template <bool SHORT>
__device__ __forceinline__ Place place(int64_t w, int u, int lane, int64_t rows, int64_t octs, int64_t segs,
                                       const Short& few) {
  const int slot = 64 * u + lane;
  Place p;
  if constexpr (SHORT) {
    const int sub = (slot * few.inv) >> 16;
    p.row = w * few.rows + sub;
    p.o = slot - sub * few.octs;
    p.ok = sub < few.rows && p.row < rows;
  } else {
    p.row = w / segs;
    p.o = (w - p.row * segs) * kSlots + slot;
    p.ok = p.row < rows && p.o < octs;
  }
  return p;
}

// Rows with unit k stride.  Wave item w: several rows (SHORT), or kSlots octets
// of row w / segs.
template <int FMT, bool SHORT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t w = wave_item();
  const int64_t rows = a.G * a.R, octs = 4 * a.Kb;
  Oct<FMT> v[kQuantU];
#pragma unroll
  for (int u = 0; u < kQuantU; ++u) {
    const Place p = place<SHORT>(w, u, lane, rows, octs, a.segs, a.few);
    const int64_t g = a.G == 1 ? 0 : p.row / a.R, r = p.row - g * a.R;
    const char* base = (const char*)a.x + (g * a.s_g + r * a.s_r) * Oct<FMT>::ES;
    v[u].load(base, 8 * p.o, p.ok ? a.K - 8 * p.o : 0);
  }
#pragma unroll
  for (int u = 0; u < kQuantU; ++u) {
    const Place p = place<SHORT>(w, u, lane, rows, octs, a.segs, a.few);
    float f[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = v[u].get(i);
      const uint32_t b = __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu;
      m = b > m ? b : m;
    }
    // the block's four lanes are neighbours: octets count from a multiple of 4
    uint32_t n = __shfl_xor(m, 1);
    m = n > m ? n : m;
    n = __shfl_xor(m, 2);
    m = n > m ? n : m;
    const uint32_t s = scale_of(m);
    if (p.ok) {
      gstore(a.data + (p.row * octs + p.o) * 4, to_codes(f, s));
      if ((p.o & 3) == 0) gstore<uint8_t>(a.scales + p.row * a.Kb + (p.o >> 2), (uint8_t)s);
    }
  }
}

// Any strides: workgroup -> 64 rows x 8 blocks, wave -> a block, lane -> a row.
// The codes change lanes through LDS, so that a store's lanes cover whole
// 128-byte lines: eight pieces of a row side by side (piece b of row r in slot
// b ^ r % 8 of the row).
constexpr int kColBlocks = 8;
template <int FMT>
__global__ __launch_bounds__(64 * kColBlocks) void quantize_columns_kernel(QuantArgs a) {
  using E = typename MxElem<FMT>::type;
  __shared__ u32x4 codes[64][kColBlocks];
  __shared__ uint8_t scales[64][kColBlocks];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t w = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, rows = a.G * a.R;
  const int64_t strip = w / a.segs, b0 = (w - strip * a.segs) * kColBlocks, b = b0 + wave;
  const int64_t row0 = strip * 64;
  if (row0 >= rows) return;
  if (row0 + lane < rows && b < a.Kb) {
    const int64_t row = row0 + lane, g = a.G == 1 ? 0 : row / a.R, r = row - g * a.R;
    const int64_t left = a.K - 32 * b;
    const int n = left < 32 ? (int)left : 32;
    const E* p = (const E*)a.x + g * a.s_g + r * a.s_r + 32 * b * a.s_k;
    E e[32];
    if (n == 32) {
#pragma unroll
      for (int i = 0; i < 32; ++i) e[i] = gload<E>(p + i * a.s_k);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) e[i] = i < n ? gload<E>(p + i * a.s_k) : (E)0;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t q = __builtin_bit_cast(uint32_t, mx_in<FMT>(e[i])) & 0x7FFFFFFFu;
      m = q > m ? q : m;
    }
    const uint32_t s = scale_of(m);
    u32x4 out;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = mx_in<FMT>(e[8 * j + i]);
      out[j] = to_codes(f, s);
    }
    codes[lane][wave ^ (lane & 7)] = out;
    scales[lane][wave] = (uint8_t)s;
  }
  __syncthreads();
  const int r = tid / kColBlocks, c = tid % kColBlocks;
  if (row0 + r < rows && b0 + c < a.Kb) {
    const int64_t at = (row0 + r) * a.Kb + b0 + c;
    store16(a.data + at * kMxBytes, codes[r][c ^ (r & 7)]);
    gstore<uint8_t>(a.scales + at, scales[r][c]);
  }
}

struct DequantArgs {
  const uint8_t* data;
  int64_t ldd;
  const uint8_t* scales;
  int64_t lds;
  int64_t R, K;
  void* y;
  int64_t ldy;     // elements
  int64_t segs;
  Short few;
};

// As quantize_rows_kernel: a lane turns 8 codes (4 bytes) into 8 elements.
template <int FMT, bool SHORT>
__global__ __launch_bounds__(256) void dequantize_kernel(DequantArgs a) {
  constexpr int ES = FMT == MX_F32 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const int64_t w = wave_item();
  const int64_t octs = (a.K + 7) / 8;
  uint32_t c[kQuantU], s[kQuantU];
#pragma unroll
  for (int u = 0; u < kQuantU; ++u) {
    const Place p = place<SHORT>(w, u, lane, a.R, octs, a.segs, a.few);
    c[u] = 0;
    if (p.ok) c[u] = gload<uint32_t>(a.data + p.row * a.ldd + 4 * p.o);
    s[u] = p.ok ? gload<uint8_t>(a.scales + p.row * a.lds + (p.o >> 2)) : 127;
  }
#pragma unroll
  for (int u = 0; u < kQuantU; ++u) {
    if constexpr (FMT == MX_F32) {
      // Half an octet is a 16-byte store: lane l takes half l % 2 of the octet
      // that lane 32 h + l / 2 loaded, so that a store's lanes lie side by side.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int from = 32 * h + lane / 2, half = lane & 1;
        const Place p = place<SHORT>(w, u, from, a.R, octs, a.segs, a.few);
        const uint32_t codes = __shfl(c[u], from) >> (16 * half);
        const bf16x8 b = mx4_to_bf16(codes, scale_f32(__shfl(s[u], from)));
        const int64_t left = p.ok ? a.K - 8 * p.o - 4 * half : 0;
        float* q = (float*)a.y + p.row * a.ldy + 8 * p.o + 4 * half;
        if (left >= 4) {
          gstore(q, f32x4{(float)b[0], (float)b[1], (float)b[2], (float)b[3]});
        } else {
#pragma unroll
          for (int i = 0; i < 3; ++i)
            if (i < left) gstore<float>(q + i, (float)b[i]);
        }
      }
      continue;
    }
    const Place p = place<SHORT>(w, u, lane, a.R, octs, a.segs, a.few);
    if (!p.ok) continue;
    const int64_t o = p.o;
    char* y = (char*)a.y + p.row * a.ldy * ES;
    const float f = scale_f32(s[u]);
    const int64_t left = a.K - 8 * o;
    char* q = y + 8 * o * ES;
    if constexpr (FMT == MX_BF16) {
      const u32x4 v = __builtin_bit_cast(u32x4, mx4_to_bf16(c[u], f));
      if (left >= 8) {
        store16(q, v);
      } else {
        for (int i = 0; i < left; ++i) gstore<uint16_t>((uint16_t*)q + i, (uint16_t)(v[i / 2] >> (16 * (i & 1))));
      }
    } else {
      // through bfloat16 (exact) and float (exact) to binary16's rounding
      const bf16x8 b = mx4_to_bf16(c[u], f);
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = (uint32_t)cvt_out<DT_F16>((float)b[2 * i]) | ((uint32_t)cvt_out<DT_F16>((float)b[2 * i + 1]) << 16);
      if (left >= 8) {
        store16(q, u32x4{h[0], h[1], h[2], h[3]});
      } else {
        for (int i = 0; i < left; ++i) gstore<uint16_t>((uint16_t*)q + i, (uint16_t)(h[i / 2] >> (16 * (i & 1))));
      }
    }
  }
}

}  // namespace gemmf16
