// The kernels of the FP8 products scaled by blocks, one translation unit for each
// pair of operand formats.
#pragma once

#include "../../include/gemm_f8_scaled.h"
#include "f8s_strip_kernel.hpp"

namespace gemmf16 {

// Those with square blocks of B (rowb = false) or row blocks; wide: through
// binary16, for float32 results.  Null where there is no such kernel.
template <int FA, int FB>
const void* f8s_fn(int variant, bool rowb, bool wide, int out);
template <> const void* f8s_fn<F8_E4M3, F8_E4M3>(int, bool, bool, int);
template <> const void* f8s_fn<F8_E4M3, F8_E5M2>(int, bool, bool, int);
template <> const void* f8s_fn<F8_E5M2, F8_E4M3>(int, bool, bool, int);
template <> const void* f8s_fn<F8_E5M2, F8_E5M2>(int, bool, bool, int);

using F8sS16x16 = F8sStrip<1, 1, 4, 8>;
using F8sS16x32 = F8sStrip<1, 2, 2, 8>;
using F8sS32x16 = F8sStrip<2, 1, 2, 8>;
using F8sS32x32 = F8sStrip<2, 2, 2, 8>;
using F8sS64x32 = F8sStrip<4, 2, 1, 8>;
using F8sS64x64 = F8sStrip<4, 4, 1, 8>;
using F8sT64x128 = F8sCfg<64, 128, 2, 2, 3>;
using F8sT128x128 = F8sCfg<128, 128, 2, 2, 2>;

// A workgroup's share of C and of K (parts: its waves' blocks of K at a time), its
// threads, how many fit a compute unit, and what it takes: per round of workgroups
// `start` and `step_full` for each `parts` blocks of K, `step` in a round that at
// most half of them fit into, either `wide` times as long through binary16
// (us; fitted to times of calls in graphs, some of which stand at plan()).
struct F8sShape {
  int rows, cols, parts, threads, per_cu;
  float start, step, step_full, wide;
};
template <class CF>
constexpr F8sShape f8s_strip_shape(float start, float step, float step_full, float wide) {
  return F8sShape{16 * CF::MT, 16 * CF::NS, CF::NW, CF::NT, 1, start, step, step_full, wide};
}
template <class CF>
constexpr F8sShape f8s_tile_shape(float start, float step, float step_full, float wide) {
  return F8sShape{CF::BM, CF::BN, 1, CF::NT, CF::PER_CU, start, step, step_full, wide};
}
constexpr F8sShape kF8sShapes[] = {
    {},
    f8s_strip_shape<F8sS16x16>(1.1f, 0.43f, 0.55f, 1.7f),
    f8s_strip_shape<F8sS16x32>(1.2f, 0.45f, 0.8f, 1.7f),
    f8s_strip_shape<F8sS32x16>(1.2f, 0.52f, 0.7f, 1.7f),
    f8s_strip_shape<F8sS32x32>(1.3f, 0.75f, 0.85f, 1.7f),
    f8s_strip_shape<F8sS64x32>(1.9f, 0.85f, 1.2f, 1.7f),
    f8s_strip_shape<F8sS64x64>(3.2f, 1.1f, 1.6f, 1.75f),
    f8s_tile_shape<F8sT64x128>(3.0f, 0.45f, 0.72f, 1.85f),
    f8s_tile_shape<F8sT128x128>(3.4f, 0.75f, 1.0f, 1.7f),
    {F8sBig::BM, F8sBig::BN, 1, F8sBig::NT, 1, 7.5f, 1.2f, 1.65f, 1.0f},
};
constexpr int kF8sVariants = sizeof(kF8sShapes) / sizeof(kF8sShapes[0]);
static_assert(kF8sVariants == GEMM_F8S_TILE_256X256 + 1, "variants of the header");

template <class CF, int FA, int FB>
const void* f8s_tile_fn(bool rowb, bool wide) {
  return rowb ? (wide ? (const void*)f8s_tile_kernel<CF, FA, FB, true, true>
                      : (const void*)f8s_tile_kernel<CF, FA, FB, true, false>)
              : (wide ? (const void*)f8s_tile_kernel<CF, FA, FB, false, true>
                      : (const void*)f8s_tile_kernel<CF, FA, FB, false, false>);
}
template <class CF, int FA, int FB>
const void* f8s_strip_fn(bool rowb, bool wide) {
  return rowb ? (wide ? (const void*)f8s_strip_kernel<CF, FA, FB, true, true>
                      : (const void*)f8s_strip_kernel<CF, FA, FB, true, false>)
              : (wide ? (const void*)f8s_strip_kernel<CF, FA, FB, false, true>
                      : (const void*)f8s_strip_kernel<CF, FA, FB, false, false>);
}

// The kernels of one format pair (in its translation unit).
#define GEMM_F8S_KERNELS(FA, FB)                                                              \
  template <>                                                                                \
  const void* f8s_fn<FA, FB>(int variant, bool rowb, bool wide, int out) {                   \
    switch (variant) {                                                                       \
      case GEMM_F8S_STRIP_16X16: return f8s_strip_fn<F8sS16x16, FA, FB>(rowb, wide);         \
      case GEMM_F8S_STRIP_16X32: return f8s_strip_fn<F8sS16x32, FA, FB>(rowb, wide);         \
      case GEMM_F8S_STRIP_32X16: return f8s_strip_fn<F8sS32x16, FA, FB>(rowb, wide);         \
      case GEMM_F8S_STRIP_32X32: return f8s_strip_fn<F8sS32x32, FA, FB>(rowb, wide);         \
      case GEMM_F8S_STRIP_64X32: return f8s_strip_fn<F8sS64x32, FA, FB>(rowb, wide);         \
      case GEMM_F8S_STRIP_64X64: return f8s_strip_fn<F8sS64x64, FA, FB>(rowb, wide);         \
      case GEMM_F8S_TILE_64X128: return f8s_tile_fn<F8sT64x128, FA, FB>(rowb, wide);         \
      case GEMM_F8S_TILE_128X128: return f8s_tile_fn<F8sT128x128, FA, FB>(rowb, wide);       \
      case GEMM_F8S_TILE_256X256:                                                            \
        if (rowb || wide) return nullptr;                                                    \
        return out == F8S_F16 ? (const void*)f8s_big_kernel<FA, FB, DT_F16>                  \
                              : (const void*)f8s_big_kernel<FA, FB, DT_BF16>;                \
    }                                                                                        \
    return nullptr;                                                                          \
  }

}  // namespace gemmf16
