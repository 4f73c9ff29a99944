// Kernel instantiations of one format pair (see f8s_tiles.hpp).
#include "f8s_tiles.hpp"

namespace gemmf16 {
GEMM_F8S_KERNELS(F8_E4M3, F8_E5M2)
}  // namespace gemmf16
