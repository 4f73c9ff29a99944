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
// 32768 x 7168 bfloat16 with a residual 276 us (6.0 TB/s), the gradients of 16384 x
// 7168 with dh 165 us (5.7 TB/s); 16 rows of 7168 3.9 us, most of it launch and latency;
// 1024 x 40000 with a residual 64 us, its gradients with dh 111.
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
  int32_t waves, lanes;    // of a row; lanes: log2 of 64, or of 16 or 32 where rows share a wave
};

// Sum over 16 neighbouring lanes, in all of them: lane exchanges that are part of
// the addition (an exchange through LDS takes some 100 cycles, and each of a
// sum's would be waited for).
__device__ __forceinline__ float sum16(float v) {
  auto other = [&](auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF,
                                                                 0xF, true));
  };
  v += other(std::integral_constant<int, 0xB1>{});    // lane ^ 1
  v += other(std::integral_constant<int, 0x4E>{});    // lane ^ 2
  v += other(std::integral_constant<int, 0x141>{});   // mirrored in 8
  v += other(std::integral_constant<int, 0x140>{});   // mirrored in 16
  return v;
}

// Sum over the wave, in all lanes.
__device__ __forceinline__ float wave_sum(float v) {
  const int s = __builtin_bit_cast(int, sum16(v));
  auto lane = [&](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(s, l)); };
  return (lane(0) + lane(16)) + (lane(32) + lane(48));
}

// Sum over the 2^lanes (16, 32 or 64) lanes of a row (or a row's part), in all of them.
__device__ __forceinline__ float row_sum(float v, int lanes) {
  if (lanes == 6) return wave_sum(v);
  v = sum16(v);
  return lanes == 5 ? v + __shfl_xor(v, 16) : v;
}

// Sum of the first n (<= 16) of 16 floats in LDS, in all lanes.
__device__ __forceinline__ float sum_parts(const float* part, int n, int lane) {
  const float v = part[lane & 15];
  return sum16((lane & 15) < n ? v : 0.0f);
}

// 8 floats -> 8 16-bit elements.
template <int FMT>
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  constexpr int DT = FMT == MX_F16 ? DT_F16 : DT_BF16;
  return u32x4{pack_out2<DT>(f[0], f[1]), pack_out2<DT>(f[2], f[3]), pack_out2<DT>(f[4], f[5]),
               pack_out2<DT>(f[6], f[7])};
}

// The first n (<= 8) of 8 16-bit elements.
template <bool ONCE = false>
__device__ __forceinline__ void store8_part(uint16_t* p, u32x4 v, int64_t n) {
  if (n >= 8) {
    gstore_once<ONCE>(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) gstore<uint16_t>(p + i, (uint16_t)(v[i / 2] >> (16 * (i % 2))));
}

// U octets of a row per lane; W32: the weight is float32, else of x's format;
// ONCE: the rows go past the caches (see kOnceBytes).
template <int FMT, int F8, int U, bool RES, bool W32, bool ONCE>
__global__ __launch_bounds__(1024) void rms_norm_f8_kernel(NormArgs a) {
  __shared__ float part[16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Row of the workgroup, wave of the row.  A workgroup of several rows has each in
  // a wave of its own, or (rows of one octet a lane) a part of one.  Other rows'
  // numbers, and with them their addresses but for 32-bit offsets, are the wave's.
  const int lanes = U > 1 ? 6 : a.lanes;
  const int share = 64 >> lanes, sub = wave / a.waves * share + (U > 1 ? 0 : lane >> lanes), rw = wave % a.waves;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / 64 / a.waves * share) + sub;
  if (row >= a.R) return;
  const int K = (int)a.K, step = 8 * 64 * a.waves, k0 = 8 * (64 * rw + (lane & ((1 << lanes) - 1)));
  constexpr uint32_t ES = 2, EW = W32 ? 4 : 2;
  // Element k0 + u step of a row, `bytes` each.
  auto at = [&](const void* base, uint32_t bytes, int u) {
    return (const char*)base + (size_t)bytes * (uint32_t)(u * step) + bytes * (uint32_t)k0;
  };
  const char* const px = (const char*)a.x + row * a.ldx * ES;
  const char* const pr = (const char*)a.residual + row * a.ldr * ES;
  char* const ph = (char*)a.h + row * a.ldh * ES;
  char* const pd = (char*)a.data + row * a.ldd;
  Oct<FMT> vx[U], vr[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = K - (k0 + u * step);
    vx[u].template load<ONCE>(at(px, ES, u), 0, n);
    if constexpr (RES) vr[u].template load<ONCE>(at(pr, ES, u), 0, n);
  }
  float v[U][8];
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = K - (k0 + u * step);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = vx[u].get(i);
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] += vr[u].get(i);
      Oct<FMT> o;
      o.v[0] = pack8<FMT>(v[u]);
      if (n > 0) store8_part<ONCE>((uint16_t*)at(ph, ES, u), o.v[0], n);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = o.get(i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(v[u][i], v[u][i], sum);
  }
  sum = row_sum(sum, lanes);
  if (a.waves > 1) {                                            // then the workgroup's only row
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    sum = sum_parts(part, a.waves, lane);
  }
  const float r = 1.0f / sqrtf(sum / (float)K + a.eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = K - (k0 + u * step);
    Oct<W32 ? MX_F32 : FMT> w;
    w.load(at(a.w, EW, u), 0, n);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[u][i] = v[u][i] * r * w.get(i);
      const uint32_t b = magnitude(v[u][i]);
      m = b > m ? b : m;
    }
    const F8Scale s = f8_scale<F8>(max16(m));
    if (n > 0) {
      store_codes<ONCE>((uint8_t*)at(pd, 1, u), f8_codes<F8>(v[u], s), n);
      if ((lane & 15) == 0) gstore<float>(a.scales + row * a.ss_r + (int64_t)((k0 + u * step) >> 7) * a.ss_k, s.scale);
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
  int32_t waves, lanes;
};

// The octet at k of a 16-bit row of K elements, zeros behind it.  One that K ends in
// (TAIL: K is no multiple of 8) is loaded from 8 before K and moved to its place by
// settle_oct when it is used, by a count that is the wave's (counts of the lanes took 6
// registers more, and with them a wave a SIMD): put together from single elements its
// wave would wait for them at once.  The gradients of 9698 x 3483 bfloat16 with dh take
// 64 us, of 9698 x 3480 52.
template <bool TAIL, bool ONCE, int FMT>
__device__ __forceinline__ void load_oct(Oct<FMT>& o, const char* row, int k, int K) {
  if (TAIL && K < 8) {
    o.load(row + 2u * (uint32_t)k, 0, K - k);
    return;
  }
  o.v[0] = zero4();
  if (k < K) o.v[0] = load16_once<ONCE>(row + 2u * (uint32_t)(!TAIL || k + 8 <= K ? k : K - 8));
}
template <bool TAIL, int FMT>
__device__ __forceinline__ void settle_oct(Oct<FMT>& o, int k, int K) {
  if (!TAIL || K < 8) return;
  const int s = 16 * (8 - K % 8);                        // bits to drop, 16 .. 112; the wave's
  const u32x4 v = o.v[0];
  const uint64_t lo = v[0] | ((uint64_t)v[1] << 32), hi = v[2] | ((uint64_t)v[3] << 32);
  const uint64_t a = s >= 64 ? hi >> (s - 64) : (lo >> s) | (hi << (64 - s)), b = s >= 64 ? 0 : hi >> s;
  if (k < K && k + 8 > K) o.v[0] = u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
}

// Rows of at most 8 waves of U octets a lane: the weight stays in registers, and
// the next row is loaded under this one's sums.  Up to two octets that takes 128
// registers at most, so four waves a SIMD; four octets take up to 256, so two.  dh is not
// loaded ahead: its registers would leave room for three waves instead of four (12000 x
// 5000 96 us instead of 89, 16384 x 7168 160 instead of 163).
constexpr int kBackThreads = 512;
template <int FMT, int U, bool TAIL, bool DH, bool W32, bool ONCE>
__global__ __launch_bounds__(kBackThreads, U > 2 ? 2 : 4) void rms_norm_back_kernel(NormBackArgs a) {
  __shared__ float part[2][2][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Only rows of one octet a lane share waves; the others' numbers, and with them
  // their addresses but for 32-bit offsets, are the wave's.
  const int lanes = U > 1 ? 6 : a.lanes;
  const int share = 64 >> lanes, sub = wave / a.waves * share + (U > 1 ? 0 : lane >> lanes), rw = wave % a.waves;
  const int64_t per = blockDim.x / 64 / a.waves * share;
  const int64_t first = (int64_t)blockIdx.x * per + sub, stride = (int64_t)gridDim.x * per;
  const int K = (int)a.K, step = 8 * 64 * a.waves, k0 = 8 * (64 * rw + (lane & ((1 << lanes) - 1)));
  constexpr uint32_t ES = 2;
  auto at = [](const void* base, uint32_t bytes) { return (const char*)base + bytes; };
  float w[U][8], dw[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = k0 + u * step;
    Oct<W32 ? MX_F32 : FMT> o;
    o.load(at(a.w, (W32 ? 4u : 2u) * k), 0, K - k);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[u][i] = o.get(i);
      dw[u][i] = 0.0f;
    }
  }
  struct Row {
    Oct<FMT> y[U], h[U];
  };
  auto load = [&](Row& r, int64_t row) {
    const char* const y = (const char*)a.dy + row * a.ldy * ES;
    const char* const h = (const char*)a.h + row * a.ldh * ES;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step;
      load_oct<TAIL, ONCE>(r.y[u], y, k, K);
      load_oct<TAIL, ONCE>(r.h[u], h, k, K);
    }
  };
  int turn = 0;
  Row next;
  if (first < a.R) load(next, first);
  for (int64_t row = first; row < a.R; row += stride, turn ^= 1) {
    Row now = next;
    Oct<FMT> dh[DH ? U : 1];
    if constexpr (DH) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * step;
        load_oct<TAIL, ONCE>(dh[u], (const char*)a.dh + row * a.lddh * ES, k, K);
      }
    }
    if (row + stride < a.R) load(next, row + stride);
    float ss = 0.0f, sg = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      settle_oct<TAIL>(now.y[u], k0 + u * step, K);
      settle_oct<TAIL>(now.h[u], k0 + u * step, K);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = now.h[u].get(i);
        ss = __builtin_fmaf(h, h, ss);
        sg = __builtin_fmaf(now.y[u].get(i) * w[u][i], h, sg);
      }
    }
    ss = row_sum(ss, lanes);
    sg = row_sum(sg, lanes);
    if (a.waves > 1) {
      // the other half of `part` is still being read by slower waves; this one was
      // before the last barrier
      if (lane == 0) {
        part[turn][0][wave] = ss;
        part[turn][1][wave] = sg;
      }
      __syncthreads();
      ss = sum_parts(part[turn][0], a.waves, lane);
      sg = sum_parts(part[turn][1], a.waves, lane);
    }
    const float r = 1.0f / sqrtf(ss / (float)a.K + a.eps);
    const float c = sg / (float)a.K * r * r;
    char* const out = (char*)a.dx + row * a.lddx * ES;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * step;
      if constexpr (DH) settle_oct<TAIL>(dh[u], k, K);
      float d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = now.h[u].get(i), y = now.y[u].get(i);
        d[i] = r * (y * w[u][i] - h * c);
        if constexpr (DH) d[i] += dh[u].get(i);
        dw[u][i] = __builtin_fmaf(y * r, h, dw[u][i]);
      }
      if (k < K) store8_part<ONCE>((uint16_t*)(out + ES * (uint32_t)k), pack8<FMT>(d), K - k);
    }
  }
  float* p = a.part + first * a.K;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = k0 + u * step;
    if (k + 8 <= K) {
      gstore<f32x4>(p + k, f32x4{dw[u][0], dw[u][1], dw[u][2], dw[u][3]});
      gstore<f32x4>(p + k + 4, f32x4{dw[u][4], dw[u][5], dw[u][6], dw[u][7]});
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (k + i < K) gstore<float>(p + k + i, dw[u][i]);
    }
  }
}

// Wider rows, up to 8 octets for each of 1024 lanes: only the weight gradient's
// sums stay in registers; a row is read again after the sums over it, from the
// caches.  Addresses are the wave's but for one offset: with one for each octet of
// each row in registers, of which there are 128 a lane, 36 to 46 of them went to memory
// (2048 x 20000 bfloat16 with dh 127 us, 113 now; 1000 x 65536 281 and 233).
constexpr int kWideThreads = 1024, kWideOcts = 8;
template <int FMT, bool DH, bool W32>
__global__ __launch_bounds__(kWideThreads) void rms_norm_back_wide_kernel(NormBackArgs a) {
  __shared__ float part[2][2][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, K = (int)a.K;
  using W = Oct<W32 ? MX_F32 : FMT>;
  constexpr uint32_t ES = 2, EW = W32 ? 4 : 2;
  // The thread's octet u of a row of elements of `bytes`: the row's part of the address
  // and u's are the wave's, so that none of them stays in a register for each octet.
  auto at = [&](const void* base, uint32_t bytes, int u) {
    return uniform_ptr((const char*)base + (size_t)bytes * (8u * kWideThreads) * (uint32_t)u) + bytes * 8u * (uint32_t)tid;
  };
  float dw[kWideOcts][8];
#pragma unroll
  for (int u = 0; u < kWideOcts; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[u][i] = 0.0f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x, turn ^= 1) {
    const char* const py = (const char*)a.dy + row * a.ldy * ES;
    const char* const ph = (const char*)a.h + row * a.ldh * ES;
    const char* const pd = (const char*)a.dh + row * a.lddh * ES;
    const char* const px = (const char*)a.dx + row * a.lddx * ES;
    float ss = 0.0f, sg = 0.0f;
    for (int u = 0; 8 * kWideThreads * u < K; ++u) {
      const int n = K - 8 * (tid + u * kWideThreads);
      Oct<FMT> y, h;
      W w;
      y.load(at(py, ES, u), 0, n);
      h.load(at(ph, ES, u), 0, n);
      w.load(at(a.w, EW, u), 0, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = __builtin_fmaf(h.get(i), h.get(i), ss);
        sg = __builtin_fmaf(y.get(i) * w.get(i), h.get(i), sg);
      }
    }
    ss = wave_sum(ss);
    sg = wave_sum(sg);
    if (lane == 0) {
      part[turn][0][wave] = ss;
      part[turn][1][wave] = sg;
    }
    __syncthreads();
    ss = sum_parts(part[turn][0], kWideThreads / 64, lane);
    sg = sum_parts(part[turn][1], kWideThreads / 64, lane);
    const float r = 1.0f / sqrtf(ss / (float)K + a.eps);
    const float c = sg / (float)K * r * r;
#pragma unroll
    for (int u = 0; u < kWideOcts; ++u) {
      asm volatile("" ::: "memory");   // no octet's loads before the one ahead is done with
      const int n = K - 8 * (tid + u * kWideThreads);
      if (n > 0) {
        Oct<FMT> y, h, d;
        W w;
        y.load(at(py, ES, u), 0, n);
        h.load(at(ph, ES, u), 0, n);
        w.load(at(a.w, EW, u), 0, n);
        if constexpr (DH) d.load(at(pd, ES, u), 0, n);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = r * (y.get(i) * w.get(i) - h.get(i) * c);
          if constexpr (DH) f[i] += d.get(i);
          dw[u][i] = __builtin_fmaf(y.get(i) * r, h.get(i), dw[u][i]);
        }
        store8_part((uint16_t*)at(px, ES, u), pack8<FMT>(f), n);
      }
    }
  }
  const char* const p = (const char*)(a.part + (int64_t)blockIdx.x * a.K);
#pragma unroll
  for (int u = 0; u < kWideOcts; ++u) {
    const int n = K - 8 * (tid + u * kWideThreads);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) gstore<float>((float*)at(p, 4, u) + i, dw[u][i]);
  }
}

// dw[k] = sum over p of part[p][k]: COLS columns a workgroup, its G = 1024 / COLS
// groups of lanes every G-th row each, eight at a time, then their sums in
// ascending order.  Few columns leave more workgroups for short rows.
template <int FMT, int COLS>
__global__ __launch_bounds__(1024) void rms_norm_dw_kernel(const float* part, int64_t parts, int64_t K, void* dw) {
  constexpr int G = 1024 / COLS;
  __shared__ float sums[G][COLS];
  const int col = threadIdx.x % COLS, group = threadIdx.x / COLS;
  const int64_t k = (int64_t)blockIdx.x * COLS + col;
  float s = 0.0f;
  if (k < K) {
    for (int64_t p = group; p < parts; p += G * 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p + G * i < parts ? gload<float>(part + (p + G * i) * K + k) : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
  }
  sums[group][col] = s;
  __syncthreads();
  if (group > 0 || k >= K) return;
#pragma unroll
  for (int i = 1; i < G; ++i) s += sums[i][col];
  if constexpr (FMT == MX_F32)
    ((float*)dw)[k] = s;
  else
    ((uint16_t*)dw)[k] = cvt_out<FMT == MX_F16 ? DT_F16 : DT_BF16>(s);
}

}  // namespace gemmf16
