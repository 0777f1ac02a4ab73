// Block-scaled GEMM: a linear backward's two products in one launch.
//
// dX = g8 . w8 (NN, a step per tile of w) and dW = g8'^T . x8' (TN, steps
// along both operands' columns) are independent; with 128 x 128 tiles of
// both in one grid the CUs that finish one's tiles start on the other's, and
// there is one launch instead of two.  Workgroups past both run the bias
// gradient's last pass (sums of the partial column sums).

#include "block_gemm_tile.hpp"

namespace fp8lin {

namespace {

constexpr int kThreads = 512, kS = 128, kStages = 4;

template <int FG, int FO>
__global__ __launch_bounds__(kThreads, 1) void block_gemm_pair_kernel(BlockTileParams dx,
                                                                     BlockTileParams dw, int n0,
                                                                     int n1, ColsumFinalJob cf) {
    constexpr int kLds0 = BlockTile<false, false, kS, kS, 4, 2, kStages>::kLds;
    constexpr int kLds1 = BlockTile<true, true, kS, kS, 4, 2, kStages>::kLds;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds0 > kLds1 ? kLds0 : kLds1];
    const int b = blockIdx.x;
    if (b < n0)
        block_gemm_tile<FG, FO, false, true, false, kS, kS, 4, 2, kStages>(dx, b, n0, smem);
    else if (b < n0 + n1)
        block_gemm_tile<FG, FO, true, true, true, kS, kS, 4, 2, kStages>(dw, b - n0, n1, smem);
    else
        colsum_final_cols<kThreads>(cf.part, cf.chunks, cf.n,
                                    (int64_t)(b - n0 - n1) * (kThreads / 4), cf.db,
                                    reinterpret_cast<float*>(smem));
}

}  // namespace

hipError_t launch_block_pair(const BlockGemmLaunch& dx, const BlockGemmLaunch& dw,
                             const ColsumFinalJob& cf, hipStream_t stream) {
    const BlockTileParams p0 = block_tile_params<kS, kS>(dx);
    BlockTileParams p1 = block_tile_params<kS, kS>(dw);
    const int n0 = p0.tiles_m * p0.tiles_n, n1 = p1.tiles_m * p1.tiles_n;
    p1.xcd_remap = p1.xcd_remap && n0 % 8 == 0;  // its ids line up with the XCDs only then
    const int extra = cf.db ? (int)((cf.n + kThreads / 4 - 1) / (kThreads / 4)) : 0;
    const dim3 grid((unsigned)(n0 + n1 + extra)), block(kThreads);
    if (dx.fmt_a == 0)
        hipLaunchKernelGGL((block_gemm_pair_kernel<0, 0>), grid, block, 0, stream, p0, p1, n0, n1, cf);
    else if (dx.fmt_b == 0)
        hipLaunchKernelGGL((block_gemm_pair_kernel<1, 0>), grid, block, 0, stream, p0, p1, n0, n1, cf);
    else
        hipLaunchKernelGGL((block_gemm_pair_kernel<1, 1>), grid, block, 0, stream, p0, p1, n0, n1, cf);
    return hipGetLastError();
}

}  // namespace fp8lin
