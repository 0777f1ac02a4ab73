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
// any address (the vector memory unit takes unaligned ones).  Where the
// matrix ends inside them, the row's last 16 are loaded instead, and shifted
// down on their way to LDS, so that no load waits for another (SHORT: rows of
// fewer than 16 bytes, gathered one by one).  kAhead stages are in flight in
// registers while one is multiplied.  Both operands' steps are per line here
// (a tile's is repeated).  Bound by the chain of a stage (LDS writes, barrier,
// LDS reads, matrix instructions, sums): 1000 x 1111 x 2047 NN 22.6 us; three or
// four stages ahead 23.9 / 24.1.
template <bool MN, int R, int NW, bool SHORT>
struct AnyOperand {
    using Op = Operand<MN, R, NW, kGroup>;
    static constexpr int kPer = Op::kPerWave;
    static constexpr int kRowsPer = MN ? 1024 / R : 8;  // stored rows a load covers
    uint4 v[kPer];

    // This lane's place in a load: stored row among its kRowsPer, first byte
    // (the same for every load of a wave).
    __device__ static void place(int wave, int lane, int& row, int& byte) {
        int c;
        Op::slot(0, wave, lane, row, c);
        row -= kRowsPer * wave;
        byte = 16 * c;
    }
    // `at`: the tile's first line at the stage's first k (uniform).  Of the
    // stage, `lines` lines and `k` of its 128 k exist.
    __device__ __forceinline__ void load(const uint8_t* at, int64_t ld, int lines, int k, int wave,
                                         int lane) {
        int row, byte;
        place(wave, lane, row, byte);
        const int rows = MN ? k : lines, width = MN ? lines : k;
        if constexpr (SHORT) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int r = kRowsPer * (wave + j * NW) + row;
                uint64_t w[2] = {0, 0};
                if (r < rows)
                    for (int i = byte; i < width && i < byte + 16; ++i)
                        w[(i - byte) / 8] |= (uint64_t)at[(int64_t)r * ld + i]
                                             << (8 * ((i - byte) % 8));
                v[j] = make_uint4((uint32_t)w[0], (uint32_t)(w[0] >> 32), (uint32_t)w[1],
                                  (uint32_t)(w[1] >> 32));
            }
        } else {
            // (offsets of a tile fit 32 bits: ld < 2^24)
            const uint32_t l = (uint32_t)ld;
            if (lines >= R && k >= kGroup) {  // uniform: all of it exists
                const uint32_t off = row * l + byte;
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    __builtin_memcpy(&v[j], at + kRowsPer * (wave + j * NW) * ld + off, 16);
            } else {
                // from 16 bytes before: a last piece may begin before this stage
                const uint32_t b = 16 + (byte + 16 <= width ? byte : width - 16);
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int r = kRowsPer * (wave + j * NW) + row;
                    __builtin_memcpy(&v[j], at - 16 + ((r < rows ? r : rows - 1) * l + b), 16);
                }
            }
        }
    }
    __device__ __forceinline__ void store(uint8_t* lds, int lines, int k, int wave, int lane) {
        const int rows = MN ? k : lines, width = MN ? lines : k;
        const bool whole = (lines >= R && k >= kGroup) || SHORT;  // uniform
        int row, byte;
        place(wave, lane, row, byte);
        if (!whole) {
            const int over = byte + 16 - width;  // bytes past the row's end
            const int bits = over <= 0 ? 0 : over >= 16 ? 128 : 8 * over;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const uint64_t w0 = v[j].x | (uint64_t)v[j].y << 32;
                const uint64_t w1 = v[j].z | (uint64_t)v[j].w << 32;
                uint64_t lo = w0, hi = w1;
                if (bits > 0 && bits < 64) lo = w0 >> bits | w1 << (64 - bits), hi = w1 >> bits;
                if (bits >= 64) lo = w1 >> (bits & 63), hi = 0;
                const bool out = bits == 128 || kRowsPer * (wave + j * NW) + row >= rows;
                v[j] = out ? make_uint4(0, 0, 0, 0)
                           : make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi,
                                        (uint32_t)(hi >> 32));
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            *reinterpret_cast<uint4*>(lds + 1024 * (wave + j * NW) + 16 * lane) = v[j];
    }
};

template <int FA, int FB, bool AMN, bool BMN, int BM, int BN, int WM, int WN, bool SHORT>
__global__ __launch_bounds__(WM* WN * 64) void block_gemm_general_kernel(BlockGemmLaunch p,
                                                                        int64_t tiles,
                                                                        int64_t tiles_n) {
    constexpr int kStage = (BM + BN) * kGroup + 4 * (BM + BN);
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
    constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, FN = TN / 32;
    static_assert(TM == 32, "one row tile per wave");
    static_assert(BM + BN <= NW * 64, "a step per lane");
    using OA = AnyOperand<AMN, BM, NW, SHORT>;
    using OB = AnyOperand<BMN, BN, NW, SHORT>;
    constexpr int kAhead = 2;
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
        } v[kAhead];
        const int arows = p.m - m0 < BM ? (int)(p.m - m0) : BM;
        const int brows = p.n - n0 < BN ? (int)(p.n - n0) : BN;
        auto k_left = [&](int64_t g) {
            const int64_t l = p.k - g * kGroup;
            return l < kGroup ? (int)l : kGroup;
        };
        auto load = [&](Stage& v, int64_t g) __attribute__((always_inline)) {
            if (g >= groups) return;
            const int64_t k0 = g * kGroup;
            v.a.load(a + (AMN ? k0 * p.lda : k0), p.lda, arows, k_left(g), wave, lane);
            v.b.load(b + (BMN ? k0 * p.ldb : k0), p.ldb, brows, k_left(g), wave, lane);
            if (step) v.s = step[g * step_k];
        };
        auto store = [&](Stage& v, int64_t g) __attribute__((always_inline)) {
            if (g >= groups) return;
            uint8_t* at = smem + (g & 1) * kStage;
            v.a.store(at, arows, k_left(g), wave, lane);
            v.b.store(at + BM * kGroup, brows, k_left(g), wave, lane);
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
        // Stage g is in LDS, the next kAhead on their way: g + 1 goes to the
        // slot that stage g - 1 left before the last barrier.
#pragma unroll
        for (int x = 0; x < kAhead; ++x) load(v[x], x);
        store(v[0], 0);
        load(v[0], kAhead);
        __syncthreads();
        for (int64_t g0 = 0; g0 < groups; g0 += kAhead) {
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const int64_t g = g0 + x;
                if (g >= groups) break;
                store(v[(x + 1) % kAhead], g + 1);
                load(v[(x + 1) % kAhead], g + 1 + kAhead);
                multiply(g);
                __syncthreads();
            }
        }
        // acc[j][e] is row wm*TM + lane%32, column wn*TN + 32j + 8*(e/4) +
        // 4*(lane/32) + e%4 of the tile: through LDS (the operands' last use is
        // behind a barrier), then out by whole rows
        constexpr int kRow = BN + 4;  // bf16 per staged row
        static_assert(BM * kRow * 2 <= 2 * kStage, "the tile fits");
        uint16_t* out = reinterpret_cast<uint16_t*>(smem);
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = wn * TN + 32 * j + 8 * q + 4 * (lane >> 5);
                float bias[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    bias[i] = p.bias && n0 + col + i < p.n ? bf16_to_f32(p.bias[n0 + col + i])
                                                           : 0.0f;
                const uint2 w = make_uint2(
                    f32x2_to_bf16x2(acc[j][4 * q] + bias[0], acc[j][4 * q + 1] + bias[1]),
                    f32x2_to_bf16x2(acc[j][4 * q + 2] + bias[2], acc[j][4 * q + 3] + bias[3]));
                *reinterpret_cast<uint2*>(out + (wm * TM + (lane & 31)) * kRow + col) = w;
            }
        __syncthreads();
        for (int row = wave; row < BM && m0 + row < p.m; row += NW)
#pragma unroll
            for (int c = lane; c < BN; c += 64)
                if (n0 + c < p.n) p.out[(m0 + row) * p.n + n0 + c] = out[row * kRow + c];
        __syncthreads();  // before the next tile's operands
    }
}

template <int FA, int FB, bool AMN, bool BMN>
hipError_t launch_general_layout(const BlockGemmLaunch& g, hipStream_t stream) {
    auto tiles = [&](int s) { return (g.m + s - 1) / s * ((g.n + s - 1) / s); };
    auto grid = [](int64_t t) { return dim3((unsigned)(t < (1 << 20) ? t : 1 << 20)); };
    // 128 x 128 tiles read half the operand bytes per output that 64 x 64 ones
    // do, once there are enough of them for every CU.
    if ((AMN ? g.m : g.k) < 16 || (BMN ? g.n : g.k) < 16)
        hipLaunchKernelGGL((block_gemm_general_kernel<FA, FB, AMN, BMN, 64, 64, 2, 2, true>),
                           grid(tiles(64)), dim3(256), 0, stream, g, tiles(64), (g.n + 63) / 64);
    else if (tiles(128) >= 256)
        hipLaunchKernelGGL((block_gemm_general_kernel<FA, FB, AMN, BMN, 128, 128, 4, 2, false>),
                           grid(tiles(128)), dim3(512), 0, stream, g, tiles(128),
                           (g.n + 127) / 128);
    else
        hipLaunchKernelGGL((block_gemm_general_kernel<FA, FB, AMN, BMN, 64, 64, 2, 2, false>),
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
    // a grid dimension counts lanes in 32 bits: fewer than 2^23 workgroups of 512
    return (double)((g.m + 127) / 128) * (double)((g.n + 127) / 128) < 8388608.0;
}

// A backward's products go in one launch of 128 x 128 tiles up to this many of
// them (two rounds of the CUs); beyond, each gains more from larger tiles.  Whole
// backward, us, one launch / each its own: 512^3 (32 tiles) 11.7 / 16.8, 2048^3
// (512) 38.8 / 43.5, 2048 x 2816 x 2048 (608) 54.3 / 53.7, 4096 x 2048 x 2048 (768)
// 62.5 / 62.5, 4096 x 4096 x 2048 (1024) 113 / 101, 4096^3 (2048) 205 / 169.
constexpr int kPairTiles = 512;

// Below this many 128 x 128 tiles, 64 x 64 ones, which spread over more CUs
// (us, 64 x 64 / 128 x 128: 1024^3 NT, 64 tiles of 128 x 128, 5.7 / 8.0;
// 1024 x 1536 x 2048, 96 tiles, NT 10.6 / 12.3, TN 14.3 / 14.2; 1920 x 2048 x
// 1024, 240 tiles, NT 13.0 / 10.1, TN 16.3 / 10.7).
constexpr int kFewTiles = 128;

// Every configuration runs one workgroup per CU, so a launch costs rounds of
// 256 tiles times a tile's time.  Those, in thousandths of a 256 x 256 tile's,
// with a step per tile of B: half as large 570, 128 x 128 350 (us, 256 x 256 /
// half / 128 x 128: 4096^3 NT 67 / 75 / 88 in one run,
// the first 68 to 71 over several cards; 3008 x 3008 x 2048 NT 31.0 / 34.9 /
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
