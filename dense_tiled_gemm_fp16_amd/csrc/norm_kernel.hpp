// Root-mean-square norm with the residual's addition, its result in FP8 by
// blocks of 128, and the norm's gradients (gfx950).
//
//   forward   h = x + residual, rounded; y = h w / sqrt(mean(h^2) + eps); y in 8
//             bits as f8s_convert.hpp has it
//   backward  with r = 1 / sqrt(mean(h^2) + eps) and g = dy w:
//             dx = r (g - h r^2 mean(g h)) + dh,   dw = sum over rows of dy h r
//
// Both are one pass over memory, which bounds them: a row stays in the
// registers of its waves between the sums over it and what is made of them.  A
// lane takes 8 consecutive elements (an octet), so that 16 neighbouring lanes
// hold a block.  Sums are float32, over a lane's elements, its wave (lane
// exchanges), its row's waves (LDS), in that order always.
//
// dw: a workgroup keeps its rows' sum for its columns in registers and leaves it
// in the workspace; a second kernel adds the workgroups' in ascending order.
#pragma once

#include "f8s_convert.hpp"

namespace gemmf16 {

struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* residual;    // or null
  int64_t ldr;
  const void* w;
  void* h;                 // with a residual
  int64_t ldh;
  uint8_t* data;
  int64_t ldd;
  float* scales;
  int64_t ss_r, ss_k;
  int64_t R, K;
  float eps;
  int32_t waves;           // of a row
};

// Sum over the wave, in all lanes.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// 8 floats -> 8 16-bit elements.
template <int FMT>
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  constexpr int DT = FMT == MX_F16 ? DT_F16 : DT_BF16;
  return u32x4{pack_out2<DT>(f[0], f[1]), pack_out2<DT>(f[2], f[3]), pack_out2<DT>(f[4], f[5]),
               pack_out2<DT>(f[6], f[7])};
}

// The first n (<= 8) of 8 16-bit elements.
__device__ __forceinline__ void store8_part(uint16_t* p, u32x4 v, int64_t n) {
  if (n >= 8) {
    store16(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) gstore<uint16_t>(p + i, (uint16_t)(v[i / 2] >> (16 * (i % 2))));
}

// U octets of a row per lane; W32: the weight is float32, else of x's format.
template <int FMT, int F8, int U, bool RES, bool W32>
__global__ __launch_bounds__(1024) void rms_norm_f8_kernel(NormArgs a) {
  __shared__ float part[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = wave / a.waves, rw = wave - sub * a.waves;    // row of the workgroup, wave of the row
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / 64 / a.waves) + sub;
  if (row >= a.R) return;                                       // several rows: each in a wave of its own
  const int step = 64 * a.waves;
  const int64_t o0 = 64 * rw + lane;
  constexpr int ES = 2;
  Oct<FMT> vx[U], vr[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t k = 8 * (o0 + u * step);
    vx[u].load((const char*)a.x + row * a.ldx * ES, k, a.K - k);
    if constexpr (RES) vr[u].load((const char*)a.residual + row * a.ldr * ES, k, a.K - k);
  }
  float v[U][8];
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = vx[u].get(i);
    if constexpr (RES) {
      const int64_t k = 8 * (o0 + u * step);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] += vr[u].get(i);
      Oct<FMT> o;
      o.v[0] = pack8<FMT>(v[u]);
      if (k < a.K) store8_part((uint16_t*)a.h + row * a.ldh + k, o.v[0], a.K - k);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = o.get(i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(v[u][i], v[u][i], sum);
  }
  sum = wave_sum(sum);
  if (a.waves > 1) {                                            // then the workgroup's only row
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int i = 0; i < a.waves; ++i) sum += part[i];
  }
  const float r = 1.0f / sqrtf(sum / (float)a.K + a.eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t k = 8 * (o0 + u * step);
    Oct<W32 ? MX_F32 : FMT> w;
    w.load(a.w, k, a.K - k);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[u][i] = v[u][i] * r * w.get(i);
      const uint32_t b = magnitude(v[u][i]);
      m = b > m ? b : m;
    }
    const F8Scale s = f8_scale<F8>(max16(m));
    if (k < a.K) {
      store_codes(a.data + row * a.ldd + k, f8_codes<F8>(v[u], s), a.K - k);
      if ((lane & 15) == 0) gstore<float>(a.scales + row * a.ss_r + (k >> 7) * a.ss_k, s.scale);
    }
  }
}

struct NormBackArgs {
  const void* dy;
  int64_t ldy;
  const void* h;
  int64_t ldh;
  const void* w;
  const void* dh;          // or null
  int64_t lddh;
  void* dx;
  int64_t lddx;
  float* part;             // [workgroups x rows of each][K]
  int64_t R, K;
  float eps;
  int32_t waves;
};

template <int FMT, int U, bool DH, bool W32>
__global__ __launch_bounds__(1024) void rms_norm_back_kernel(NormBackArgs a) {
  __shared__ float part[2][2][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = wave / a.waves, rw = wave - sub * a.waves;
  const int64_t per = blockDim.x / 64 / a.waves;
  const int64_t first = (int64_t)blockIdx.x * per + sub, stride = (int64_t)gridDim.x * per;
  const int step = 64 * a.waves;
  const int64_t o0 = 64 * rw + lane;
  constexpr int ES = 2;
  float w[U][8], dw[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t k = 8 * (o0 + u * step);
    Oct<W32 ? MX_F32 : FMT> o;
    o.load(a.w, k, a.K - k);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[u][i] = o.get(i);
      dw[u][i] = 0.0f;
    }
  }
  int turn = 0;
  for (int64_t row = first; row < a.R; row += stride, turn ^= 1) {
    Oct<FMT> vy[U], vh[U], vd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = 8 * (o0 + u * step);
      vy[u].load((const char*)a.dy + row * a.ldy * ES, k, a.K - k);
      vh[u].load((const char*)a.h + row * a.ldh * ES, k, a.K - k);
      if constexpr (DH) vd[u].load((const char*)a.dh + row * a.lddh * ES, k, a.K - k);
    }
    float ss = 0.0f, sg = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = vh[u].get(i);
        ss = __builtin_fmaf(h, h, ss);
        sg = __builtin_fmaf(vy[u].get(i) * w[u][i], h, sg);
      }
    ss = wave_sum(ss);
    sg = wave_sum(sg);
    if (a.waves > 1) {
      // the other half of `part` is still being read by slower waves; this one was
      // before the last barrier
      if (lane == 0) {
        part[turn][0][wave] = ss;
        part[turn][1][wave] = sg;
      }
      __syncthreads();
      ss = sg = 0.0f;
      for (int i = 0; i < a.waves; ++i) {
        ss += part[turn][0][i];
        sg += part[turn][1][i];
      }
    }
    const float r = 1.0f / sqrtf(ss / (float)a.K + a.eps);
    const float c = sg / (float)a.K * r * r;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = 8 * (o0 + u * step);
      float d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = vh[u].get(i), y = vy[u].get(i);
        d[i] = r * (y * w[u][i] - h * c);
        if constexpr (DH) d[i] += vd[u].get(i);
        dw[u][i] = __builtin_fmaf(y * r, h, dw[u][i]);
      }
      if (k < a.K) store8_part((uint16_t*)a.dx + row * a.lddx + k, pack8<FMT>(d), a.K - k);
    }
  }
  float* p = a.part + first * a.K;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t k = 8 * (o0 + u * step);
    if (k + 8 <= a.K) {
      gstore<f32x4>(p + k, f32x4{dw[u][0], dw[u][1], dw[u][2], dw[u][3]});
      gstore<f32x4>(p + k + 4, f32x4{dw[u][4], dw[u][5], dw[u][6], dw[u][7]});
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (k + i < a.K) gstore<float>(p + k + i, dw[u][i]);
    }
  }
}

// dw[k] = sum over p of part[p][k]: 64 columns a workgroup, its 16 waves every
// 16th row each, then their sums in ascending order.
template <int FMT>
__global__ __launch_bounds__(1024) void rms_norm_dw_kernel(const float* part, int64_t parts, int64_t K, void* dw) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (k < K)
    for (int64_t p = wave; p < parts; p += 16) s += part[p * K + k];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave > 0 || k >= K) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += sums[i][lane];
  if constexpr (FMT == MX_F32)
    ((float*)dw)[k] = s;
  else
    ((uint16_t*)dw)[k] = cvt_out<FMT == MX_F16 ? DT_F16 : DT_BF16>(s);
}

}  // namespace gemmf16
