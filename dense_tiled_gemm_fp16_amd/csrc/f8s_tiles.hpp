// The tiles of the FP8 products scaled by blocks, one translation unit for each
// pair of operand formats.
#pragma once

#include "f8s_tile_kernel.hpp"

namespace gemmf16 {

enum F8sTile { F8S_TILE_128 = 0 };

using F8sT128 = F8sCfg<128, 128, 2, 2, 4>;

template <int FA, int FB>
const void* f8s_tile_of(int tile, bool rowb);

template <> const void* f8s_tile_of<F8_E4M3, F8_E4M3>(int, bool);
template <> const void* f8s_tile_of<F8_E4M3, F8_E5M2>(int, bool);
template <> const void* f8s_tile_of<F8_E5M2, F8_E4M3>(int, bool);
template <> const void* f8s_tile_of<F8_E5M2, F8_E5M2>(int, bool);


inline const void* f8s_tile_fn(int tile, int fa, int fb, bool rowb) {
  if (fa == 0) return fb == 0 ? f8s_tile_of<F8_E4M3, F8_E4M3>(tile, rowb) : f8s_tile_of<F8_E4M3, F8_E5M2>(tile, rowb);
  return fb == 0 ? f8s_tile_of<F8_E5M2, F8_E4M3>(tile, rowb) : f8s_tile_of<F8_E5M2, F8_E5M2>(tile, rowb);
}

// Kernel addresses of one format pair (in its translation unit).
#define GEMM_F8S_TILES(FA, FB)                                                                             \
  template <>                                                                                             \
  const void* f8s_tile_of<FA, FB>(int, bool rowb) {                                                       \
    return rowb ? (const void*)f8s_tile_kernel<F8sT128, FA, FB, true>                                     \
                : (const void*)f8s_tile_kernel<F8sT128, FA, FB, false>;                                   \
  }

}  // namespace gemmf16
