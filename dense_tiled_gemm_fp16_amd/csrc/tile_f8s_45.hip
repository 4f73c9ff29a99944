#include "f8s_tiles.hpp"

namespace gemmf16 {
GEMM_F8S_TILES(F8_E4M3, F8_E5M2)
}  // namespace gemmf16
