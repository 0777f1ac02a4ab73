// Block-scaled fp8 product:
//   out[i][j] = bf16( sum_kb sa(i, kb) sb(kb, j) * sum_{k in group kb} A[i][k] B[k][j] + bias[j] )
// with fp32 sums.  The sum over one group of 128 k is what the matrix
// instruction gives from a zero accumulator; it is then scaled by the
// product of the two steps and added to the running sum (one rounding of
// the product of the steps, one fused multiply-add per group).
//
// This file holds the dispatcher and the general kernel (the tiled kernels
// are block_gemm_tile.hpp's), which takes any
// layout, size, stride and alignment: every lane gathers its operand bytes
// one by one and each wave owns a 16 x 16 output tile, whose 16x16x128
// matrix instruction covers exactly one group of k.

#include "block.hpp"
#include "block_gemm_tile.hpp"
#include "common.hpp"

namespace fp8lin {

namespace {

constexpr int kGenThreads = 256;  // 4 waves, 2 x 2 grid of 16 x 16 tiles

__device__ __forceinline__ float scale_at(const BlockScale& s, int64_t i, int64_t kb) {
    return s.s[(i >> s.shift) * s.si + kb * s.sk];
}

template <int FA, int FB>
__global__ __launch_bounds__(kGenThreads) void block_gemm_general_kernel(BlockGemmLaunch p) {
    const int lane = threadIdx.x % kWave;
    const int wave = threadIdx.x / kWave;
    const int64_t col0 = (int64_t)blockIdx.x * 32 + (wave % 2) * 16;
    const int64_t bc = col0 + lane % 16;  // this lane's column of B and of the output
    const int kq = 32 * (lane / 16);
    for (int64_t by = blockIdx.y; by * 32 < p.m; by += gridDim.y) {
        const int64_t row0 = by * 32 + (wave / 2) * 16;
        const int64_t ar = row0 + lane % 16;  // this lane's row of A
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t k0 = 0, kb = 0; k0 < p.k; k0 += kGroup, ++kb) {
            union {
                v8i v;
                uint8_t b[32];
            } xa, xb;
#pragma unroll 4
            for (int j = 0; j < 32; ++j) {
                const int64_t kk = k0 + kq + j;
                uint8_t va = 0, vb = 0;
                if (kk < p.k) {
                    if (ar < p.m) va = p.trans_a ? p.a[kk * p.lda + ar] : p.a[ar * p.lda + kk];
                    if (bc < p.n) vb = p.trans_b ? p.b[bc * p.ldb + kk] : p.b[kk * p.ldb + bc];
                }
                xa.b[j] = va;
                xb.b[j] = vb;
            }
            const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                xa.v, xb.v, v4f{0.0f, 0.0f, 0.0f, 0.0f}, FA, FB, 0, 0, 0, 0);
            const float sb = bc < p.n ? scale_at(p.sb, bc, kb) : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t r = row0 + 4 * (lane / 16) + i;
                const float sa = r < p.m ? scale_at(p.sa, r, kb) : 0.0f;
                acc[i] = fmaf(part[i], sa * sb, acc[i]);
            }
        }
        if (bc >= p.n) continue;
        const float bias = p.bias ? bf16_to_f32(p.bias[bc]) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = row0 + 4 * (lane / 16) + i;
            if (r < p.m) p.out[r * p.n + bc] = f32_to_bf16(acc[i] + bias);
        }
    }
}

template <int FA, int FB>
hipError_t launch_general(const BlockGemmLaunch& g, hipStream_t stream) {
    const int64_t gy = (g.m + 31) / 32;
    const dim3 grid((unsigned)((g.n + 31) / 32), (unsigned)(gy < 65535 ? gy : 65535));
    hipLaunchKernelGGL((block_gemm_general_kernel<FA, FB>), grid, dim3(kGenThreads), 0, stream, g);
    return hipGetLastError();
}

}  // namespace

size_t block_gemm_workspace(int64_t, int64_t, int64_t) { return 0; }

// What the tiled kernels take: 16-byte aligned operands and leading
// dimensions, whole 16-byte pieces along the contiguous dimension, operands
// that 32-bit offsets reach.
static bool tiled_supported(const BlockGemmLaunch& g) {
    if (g.fmt_a == 0 && g.fmt_b == 1) return false;
    if (g.trans_a && g.trans_b) return false;
    if ((reinterpret_cast<uintptr_t>(g.a) | reinterpret_cast<uintptr_t>(g.b)) & 15) return false;
    if (g.lda % 16 || g.ldb % 16) return false;
    if ((g.trans_a ? g.m : g.k) % 16 || (g.trans_b ? g.k : g.n) % 16) return false;
    const double lim = 2147483647.0;
    if ((double)(g.trans_a ? g.k : g.m) * (double)g.lda >= lim) return false;
    if ((double)(g.trans_b ? g.n : g.k) * (double)g.ldb >= lim) return false;
    if ((double)g.sa.sk >= lim / 4 || (double)g.sb.sk >= lim / 4) return false;
    return (double)((g.m + 127) / 128) * (double)((g.n + 127) / 128) < lim;
}

static BlockCfg tile_cfg(const BlockGemmLaunch& g) {
    auto rounds = [&](int bm, int bn) {
        return (((g.m + bm - 1) / bm) * ((g.n + bn - 1) / bn) + 255) / 256;
    };
    const BlockCfg half = g.n >= g.m ? BlockCfg::kWide : BlockCfg::kTall;
    const int64_t half_rounds = g.n >= g.m ? rounds(128, 256) : rounds(256, 128);
    return half_rounds * 675 <= rounds(128, 128) * 475 ? half : BlockCfg::kMid;
}

hipError_t launch_block_gemm(const BlockGemmLaunch& g, hipStream_t stream) {
    if (tiled_supported(g)) {
        const bool bvec = g.sb.shift == 0;
        const BlockCfg c = tile_cfg(g);
        if (g.trans_a) return launch_block_tn(g, bvec, c, stream);
        return g.trans_b ? launch_block_nt(g, bvec, c, stream) : launch_block_nn(g, bvec, c, stream);
    }
    if (g.fmt_a == 0) return g.fmt_b == 0 ? launch_general<0, 0>(g, stream)
                                          : launch_general<0, 1>(g, stream);
    return g.fmt_b == 0 ? launch_general<1, 0>(g, stream) : launch_general<1, 1>(g, stream);
}

}  // namespace fp8lin
