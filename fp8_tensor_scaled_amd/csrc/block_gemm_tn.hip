// Block-scaled GEMM, TN instances.
#include "block_gemm_tile.hpp"

namespace fp8lin {

hipError_t launch_block_tn(const BlockGemmLaunch& g, bool bvec, BlockCfg c, hipStream_t stream) {
    return launch_block_layout<true, true>(g, bvec, c, stream);
}

}  // namespace fp8lin
