// Block-scaled fp8 product:
//   out[i][j] = bf16( sum_kb sa(i, kb) sb(kb, j) * sum_{k in group kb} A[i][k] B[k][j] + bias[j] )
// with fp32 sums.  The sum over one group of 128 k is what the matrix
// instruction gives from a zero accumulator; it is then scaled by the
// product of the two steps and added to the running sum (one rounding of
// the product of the steps, one fused multiply-add per group).
//
// This file holds the dispatcher and the general kernel, which takes any
// layout, size, stride and alignment (the tiled kernels, for operands of
// whole 16-byte pieces, are block_gemm_tile.hpp's).

#include "block.hpp"
#include "block_gemm_tile.hpp"
#include "common.hpp"

namespace fp8lin {

namespace {

// The general kernel: two LDS stages of one group of k in the tiled kernels'
// layout.  Operands come through registers: a lane's 16 bytes may begin at
// any address (the vector memory unit takes unaligned ones); where the
// matrix ends inside them, the row's last 16 are loaded and shifted down.
// Two stages are in flight in registers while one is multiplied.  Both
// operands' steps are per line here (a tile's is repeated), and all offsets
// are 64-bit.
template <bool MN, int R, int NW>
struct AnyOperand {
    using Op = Operand<MN, R, NW, kGroup>;
    static constexpr int kPer = Op::kPerWave;
    uint4 v[kPer];

    // The stage at k0: `base` is the operand at this tile's first line.
    __device__ void load(const uint8_t* base, int64_t ld, int64_t lines, int64_t k0, int64_t k,
                         int wave, int lane) {
        const int64_t rows = MN ? k : lines, width = MN ? lines : k;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            int row, c;
            Op::slot(j, wave, lane, row, c);
            const int64_t across = MN ? k0 + row : row;       // which stored row
            const int64_t along = MN ? 16 * c : k0 + 16 * c;  // first byte in it
            v[j] = make_uint4(0, 0, 0, 0);
            if (across >= rows || along >= width) continue;
            const uint8_t* src = base + across * ld;
            const int64_t over = along + 16 - width;  // bytes past the row's end
            if (over <= 0) {
                __builtin_memcpy(&v[j], src + along, 16);
            } else if (width >= 16) {
                uint64_t w[2];
                __builtin_memcpy(w, src + width - 16, 16);
                const int bits = 8 * (int)over;  // 8 .. 120
                const uint64_t lo = bits < 64 ? w[0] >> bits | w[1] << (64 - bits)
                                              : w[1] >> (bits - 64);
                const uint64_t hi = bits < 64 ? w[1] >> bits : 0;
                v[j] = make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi,
                                  (uint32_t)(hi >> 32));
            } else {  // the whole row is shorter
                uint64_t w[2] = {0, 0};
                for (int i = 0; i < width; ++i)
                    w[i / 8] |= (uint64_t)src[along + i] << (8 * (i % 8));
                v[j] = make_uint4((uint32_t)w[0], (uint32_t)(w[0] >> 32), (uint32_t)w[1],
                                  (uint32_t)(w[1] >> 32));
            }
        }
    }
    __device__ void store(uint8_t* lds, int wave, int lane) const {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            *reinterpret_cast<uint4*>(lds + 1024 * (wave + j * NW) + 16 * lane) = v[j];
    }
};

template <int FA, int FB, bool AMN, bool BMN, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void block_gemm_general_kernel(BlockGemmLaunch p,
                                                                        int64_t tiles,
                                                                        int64_t tiles_n) {
    constexpr int kStage = (BM + BN) * kGroup + 4 * (BM + BN);
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
    constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, FN = TN / 32;
    static_assert(TM == 32, "one row tile per wave");
    static_assert(BM + BN <= NW * 64, "a step per lane");
    using OA = AnyOperand<AMN, BM, NW>;
    using OB = AnyOperand<BMN, BN, NW>;
    constexpr int kRowA = AMN ? 0 : kGroup, kRowB = BMN ? 0 : kGroup;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int64_t groups = (p.k + kGroup - 1) / kGroup;
    const uint32_t aoff = OA::Op::frag_off(AMN ? wm * TM : 0, lane);
    uint32_t boff[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) boff[j] = OB::Op::frag_off(BMN ? wn * TN + 32 * j : 0, lane);

    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t m0 = tile / tiles_n * BM, n0 = tile % tiles_n * BN;
        const uint8_t* a = p.a + (AMN ? m0 : m0 * p.lda);
        const uint8_t* b = p.b + (BMN ? n0 : n0 * p.ldb);
        // lane e carries a step: row e's, then column e - BM's
        const int e = threadIdx.x;
        const float* step = nullptr;
        int64_t step_k = 0;
        if (e < BM && m0 + e < p.m) {
            step = p.sa.s + ((m0 + e) >> p.sa.shift) * p.sa.si;
            step_k = p.sa.sk;
        } else if (e >= BM && e < BM + BN && n0 + e - BM < p.n) {
            step = p.sb.s + ((n0 + e - BM) >> p.sb.shift) * p.sb.si;
            step_k = p.sb.sk;
        }
        struct Stage {
            OA a;
            OB b;
            float s = 0.0f;
        } one, two;
        auto load = [&](Stage& v, int64_t g) __attribute__((always_inline)) {
            if (g >= groups) return;
            v.a.load(a, p.lda, p.m - m0, g * kGroup, p.k, wave, lane);
            v.b.load(b, p.ldb, p.n - n0, g * kGroup, p.k, wave, lane);
            if (step) v.s = step[g * step_k];
        };
        auto store = [&](const Stage& v, int64_t g) __attribute__((always_inline)) {
            if (g >= groups) return;
            uint8_t* at = smem + (g & 1) * kStage;
            v.a.store(at, wave, lane);
            v.b.store(at + BM * kGroup, wave, lane);
            if (e < BM + BN) *reinterpret_cast<float*>(at + (BM + BN) * kGroup + 4 * e) = v.s;
        };
        v16f acc[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[j][i] = 0.0f;
        auto multiply = [&](int64_t g) __attribute__((always_inline)) {
            uint8_t* at = smem + (g & 1) * kStage;
            const uint8_t* la = at + wm * TM * kRowA;
            const uint8_t* lb = at + BM * kGroup + wn * TN * kRowB;
            const float* ls = reinterpret_cast<const float*>(at + (BM + BN) * kGroup);
            const v8i a0 = OA::Op::template frag<0>(la, aoff);
            const v8i a1 = OA::Op::template frag<1>(la, aoff);
            const float sa = ls[wm * TM + (lane & 31)];
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                v16f part = {0};
                part = mfma_ba<FA, FB>(OB::Op::template frag<0>(lb + 32 * j * kRowB, boff[j]), a0,
                                       part);
                part = mfma_ba<FA, FB>(OB::Op::template frag<1>(lb + 32 * j * kRowB, boff[j]), a1,
                                       part);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v4f sb = *reinterpret_cast<const v4f*>(
                        ls + BM + wn * TN + 32 * j + 8 * q + 4 * (lane >> 5));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[j][4 * q + i] = fmaf(part[4 * q + i] * sa, sb[i], acc[j][4 * q + i]);
                }
            }
        };
        // Stage g is in LDS, g + 1 in `next` and g + 2 on its way: `next` goes
        // to the slot that stage g - 1 left before the last barrier.
        auto turn = [&](Stage& next, int64_t g) __attribute__((always_inline)) {
            store(next, g + 1);
            load(next, g + 3);
            multiply(g);
            __syncthreads();
        };
        load(one, 0);
        load(two, 1);
        store(one, 0);
        load(one, 2);
        __syncthreads();
        for (int64_t g = 0; g < groups; g += 2) {
            turn(two, g);
            if (g + 1 < groups) turn(one, g + 1);
        }
        // acc[j][e] is row m0 + wm*TM + lane%32, column n0 + wn*TN + 32j +
        // 8*(e/4) + 4*(lane/32) + e%4
        const int64_t gm = m0 + wm * TM + (lane & 31);
        if (gm < p.m) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int64_t gn =
                        n0 + wn * TN + 32 * j + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
                    if (gn < p.n) {
                        const float bias = p.bias ? bf16_to_f32(p.bias[gn]) : 0.0f;
                        p.out[gm * p.n + gn] = f32_to_bf16(acc[j][i] + bias);
                    }
                }
        }
    }
}

template <int FA, int FB, bool AMN, bool BMN>
hipError_t launch_general_layout(const BlockGemmLaunch& g, hipStream_t stream) {
    auto tiles = [&](int s) { return (g.m + s - 1) / s * ((g.n + s - 1) / s); };
    auto grid = [](int64_t t) { return dim3((unsigned)(t < (1 << 20) ? t : 1 << 20)); };
    // 128 x 128 tiles read half the operand bytes per output that 64 x 64 ones
    // do, once there are enough of them for every CU.
    if (tiles(128) >= 256)
        hipLaunchKernelGGL((block_gemm_general_kernel<FA, FB, AMN, BMN, 128, 128, 4, 2>),
                           grid(tiles(128)), dim3(512), 0, stream, g, tiles(128),
                           (g.n + 127) / 128);
    else
        hipLaunchKernelGGL((block_gemm_general_kernel<FA, FB, AMN, BMN, 64, 64, 2, 2>),
                           grid(tiles(64)), dim3(256), 0, stream, g, tiles(64), (g.n + 63) / 64);
    return hipGetLastError();
}

template <int FA, int FB>
hipError_t launch_general(const BlockGemmLaunch& g, hipStream_t stream) {
    const bool am = g.trans_a != 0, bm = g.trans_b == 0;
    if (am) return bm ? launch_general_layout<FA, FB, true, true>(g, stream)
                      : launch_general_layout<FA, FB, true, false>(g, stream);
    return bm ? launch_general_layout<FA, FB, false, true>(g, stream)
              : launch_general_layout<FA, FB, false, false>(g, stream);
}

}  // namespace

// Shares of a tile along k.  A group of k takes a 64 x 64 tile's workgroup
// about 0.27 us (a chain of LDS reads, matrix instructions and a barrier); joining s
// shares measured 2.5 us + 0.35 us s.  The cheapest number that gives each
// CU at most one workgroup.
int block_gemm_splits(int64_t m, int64_t n, int64_t k) {
    const double all = (double)((m + 63) / 64) * (double)((n + 63) / 64);
    if (all > 128) return 1;
    const int tiles = (int)all;
    const int64_t groups = groups_of(k);
    int64_t best = 1, cost = 27 * groups;
    for (int64_t s = 2; s <= 16 && s * tiles <= 256; ++s) {
        const int64_t per = (groups + s - 1) / s;
        if ((groups + per - 1) / per != s) continue;  // a share would be empty
        const int64_t c = 27 * per + 250 + 35 * s;
        if (c < cost) cost = c, best = s;
    }
    return (int)best;
}

size_t block_gemm_partials(int64_t m, int64_t n, int64_t k) {
    const int s = block_gemm_splits(m, n, k);
    if (s == 1) return 0;
    return (size_t)s * ((m + 63) / 64) * ((n + 63) / 64) * 64 * 64 * sizeof(float);
}

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
    return (double)((g.m + 63) / 64) * (double)((g.n + 63) / 64) < lim;
}

// A backward's products go in one launch of 128 x 128 tiles up to this many of
// them (four rounds of the CUs); beyond, each gains more from larger tiles.
constexpr int kPairTiles = 1024;

// Below this many 128 x 128 tiles, 64 x 64 ones, which spread over more CUs
// (us, 64 x 64 / 128 x 128: 1024^3 NT, 64 tiles of 128 x 128, 5.7 / 8.0;
// 1024 x 1536 x 2048, 96 tiles, NT 10.6 / 12.3, TN 14.3 / 14.2; 1920 x 2048 x
// 1024, 240 tiles, NT 13.0 / 10.1, TN 16.3 / 10.7).
constexpr int kFewTiles = 128;

// Every configuration runs one workgroup per CU, so a launch costs rounds of
// 256 tiles times a tile's time.  Those, in thousandths of a 256 x 256 tile's,
// with a step per tile of B: half as large 570, 128 x 128 350 (us, 256 x 256 /
// half / 128 x 128: 4096^3 NT 67 / 75 / 88; 3008 x 3008 x 2048 NT 31.0 / 34.9 /
// 35.5; 2048 x 4096 x 4096 NT 54.5 / 38.9 / 44.7; 2048^3 NT - / 17.4 / 15.2).
// With a step per column of B, which the 256 x 256 tile has no registers for, a
// 128 x 128 one costs 475 / 675 of the half (2048^3 TN 21.2 / 16.5, 3008 x 3008 x
// 1024 TN 26.4 / 27.9).
static BlockCfg tile_cfg(const BlockGemmLaunch& g) {
    auto tiles = [&](int bm, int bn) { return ((g.m + bm - 1) / bm) * ((g.n + bn - 1) / bn); };
    auto rounds = [&](int bm, int bn) { return (tiles(bm, bn) + 255) / 256; };
    if (tiles(128, 128) < kFewTiles) return BlockCfg::kSmall;
    const bool bvec = g.sb.shift == 0;
    const BlockCfg half = g.n >= g.m ? BlockCfg::kWide : BlockCfg::kTall;
    const int64_t half_cost =
        (g.n >= g.m ? rounds(128, 256) : rounds(256, 128)) * (bvec ? 675 : 570);
    const int64_t mid_cost = rounds(128, 128) * (bvec ? 475 : 350);
    if (!bvec && rounds(256, 256) * 1000 <= half_cost && rounds(256, 256) * 1000 <= mid_cost)
        return BlockCfg::kBig;
    return half_cost <= mid_cost ? half : BlockCfg::kMid;
}

hipError_t launch_block_gemm_pair(const BlockGemmLaunch& dx, const BlockGemmLaunch& dw,
                                  const ColsumFinalJob& cf, hipStream_t stream) {
    auto tiles = [](const BlockGemmLaunch& g) {
        return (double)((g.m + 127) / 128) * (double)((g.n + 127) / 128);
    };
    if (tiled_supported(dx) && tiled_supported(dw) && dx.fmt_b == dw.fmt_b &&
        dx.fmt_a == dw.fmt_a && dx.sb.shift != 0 && dw.sb.shift == 0 &&
        tiles(dx) + tiles(dw) <= kPairTiles)
        return launch_block_pair(dx, dw, cf, stream);
    hipError_t e = launch_block_gemm(dx, stream);
    if (e == hipSuccess) e = launch_block_gemm(dw, stream);
    if (e == hipSuccess && cf.db) e = launch_colsum_final_job(cf, stream);
    return e;
}

hipError_t launch_block_gemm(const BlockGemmLaunch& g, hipStream_t stream) {
    if (tiled_supported(g)) {
        // Short A against a weight: the bandwidth-shaped kernel, but for a long k
        // over few columns, where the split one has more of the chip to itself
        // (16 x 128 x 16384: 11.6 us split, 22.5; 16 x 1024 x 4096: 8.0 against 9.2).
        if (!g.trans_a && g.trans_b && g.m <= 64 &&
            (g.k <= 64 * kGroup || !g.part || block_gemm_splits(g.m, g.n, g.k) == 1))
            return launch_block_skinny(g, stream);
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
