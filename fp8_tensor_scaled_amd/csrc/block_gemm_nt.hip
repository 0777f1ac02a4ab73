// Block-scaled GEMM, NT instances.
#include "block_gemm_tile.hpp"

namespace fp8lin {

hipError_t launch_block_nt(const BlockGemmLaunch& g, bool bvec, BlockCfg c, hipStream_t stream) {
    return launch_block_layout<false, false>(g, bvec, c, stream);
}

}  // namespace fp8lin
