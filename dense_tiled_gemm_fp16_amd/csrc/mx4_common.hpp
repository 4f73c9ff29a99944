// Device helpers for MX FP4 (gfx950): 4-bit codes and block scales in
// registers.
//
// A block of 32 codes is 16 bytes: one lane's operand of the 4-bit matrix
// instructions, and what one 16-byte load brings.  The packed converts
// (v_cvt_scalef32_pk_*) work on one byte = two codes at a time; the code to
// bfloat16 convert is exact for every scale byte (measured over all 256 x 16,
// subnormal scales and the NaN scale included; values of 2^128 and more, at scale
// bytes 253 and 254, become infinite), the one to binary16 for scale bytes 104 ..
// 140 and, below 61, gives zeros.
#pragma once

#include <cstring>

#include "tile_common.hpp"

namespace gemmf16 {

constexpr int kMxBlock = 32;    // elements that share a scale
constexpr int kMxBytes = 16;    // their codes

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Loads and stores of global memory at any alignment (the hardware takes
// unaligned addresses; aligned ones cost nothing extra).  The address space is
// named, because a pointer that went through integers or structures is taken
// for a generic one: a flat instruction then also counts with the LDS, and
// every wait for an LDS read waits for all loads in flight.
#define GEMM_GLOBAL __attribute__((address_space(1)))
template <class T>
__device__ __forceinline__ T gload(const void* p) {
  typedef T Any __attribute__((aligned(1)));
  return *(const GEMM_GLOBAL Any*)p;
}
template <class T>
__device__ __forceinline__ void gstore(void* p, T v) {
  typedef T Any __attribute__((aligned(1)));
  *(GEMM_GLOBAL Any*)p = v;
}
__device__ __forceinline__ u32x4 load16(const void* p) { return gload<u32x4>(p); }
__device__ __forceinline__ void store16(void* p, u32x4 v) { gstore<u32x4>(p, v); }

// The same for what is read or written once and too much for the last cache to
// keep (kOnceBytes): past the caches.
template <bool ONCE>
__device__ __forceinline__ u32x4 load16_once(const void* p) {
  typedef u32x4 Any __attribute__((aligned(1)));
  if constexpr (ONCE) return __builtin_nontemporal_load((const GEMM_GLOBAL Any*)p);
  return load16(p);
}
template <bool ONCE, class T>
__device__ __forceinline__ void gstore_once(void* p, T v) {
  typedef T Any __attribute__((aligned(1)));
  if constexpr (ONCE)
    __builtin_nontemporal_store(v, (GEMM_GLOBAL Any*)p);
  else
    gstore<T>(p, v);
}

// v without its lowest `bytes` (1 .. 15), zeros from above.
__device__ __forceinline__ u32x4 drop_bytes(u32x4 v, int bytes) {
  uint64_t lo = (uint64_t)v[0] | (uint64_t)v[1] << 32, hi = (uint64_t)v[2] | (uint64_t)v[3] << 32;
  if (bytes >= 8) {
    lo = hi;
    hi = 0;
    bytes -= 8;
  }
  if (bytes > 0) {
    lo = lo >> (8 * bytes) | hi << (64 - 8 * bytes);
    hi >>= 8 * bytes;
  }
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Bytes at .. at + 15 of a row, the first n of them, zeros behind (n is the rest
// of the row where it is below 16).  The rest comes by one load of the row's
// last 16 bytes: byte by byte, each load's latency is waited for.
__device__ __forceinline__ u32x4 load_bytes(const char* row, int64_t at, int64_t n) {
  if (n >= 16) return load16(row + at);
  if (n <= 0) return zero4();
  if (at + n >= 16) return drop_bytes(load16(row + at + n - 16), 16 - (int)n);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 15; ++e)
    if (e < n) w[e / 4] |= (uint32_t)gload<uint8_t>(row + at + e) << (8 * (e % 4));
  return u32x4{w[0], w[1], w[2], w[3]};
}

// n (1, 2 or 4) dwords.
template <int N>
__device__ __forceinline__ void load_dwords(uint32_t (&d)[N], const void* p) {
  if constexpr (N == 4) {
    const u32x4 v = gload<u32x4>(p);
    d[0] = v[0]; d[1] = v[1]; d[2] = v[2]; d[3] = v[3];
  } else if constexpr (N == 2) {
    const u32x2 v = gload<u32x2>(p);
    d[0] = v[0]; d[1] = v[1];
  } else {
    static_assert(N == 1, "1, 2 or 4");
    d[0] = gload<uint32_t>(p);
  }
}

// A scale byte as the float whose exponent the converts use.
__device__ __forceinline__ float scale_f32(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// The 8 codes of a dword times the scale, as binary16 or bfloat16.
__device__ __forceinline__ f16x8 mx4_to_f16(uint32_t d, float s) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, s, 0);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, s, 1);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, s, 2);
  const f16x2 e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, s, 3);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}
__device__ __forceinline__ bf16x8 mx4_to_bf16(uint32_t d, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// Codes k .. of a 16-byte block kept where k < nvalid (0 .. 32), zero codes
// from there on.
__device__ __forceinline__ u32x4 mask_codes(u32x4 v, int nvalid) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = nvalid - 8 * j;
    v[j] = n >= 8 ? v[j] : (n <= 0 ? 0u : (v[j] & ((1u << (4 * n)) - 1u)));
  }
  return v;
}

}  // namespace gemmf16
