// Block-scaled fp8 GEMM for short A (m <= 64), both operands k-contiguous
// (NT): what a few decoded tokens multiply with a weight, bound by reading B.
//
//  * One workgroup of 8 waves owns all m rows x 32 columns; B's rows are
//    spread so that each XCD streams a contiguous slab of it.
//  * Operands go global -> LDS in chunks of 512 k, two whole 512-byte row
//    segments per load instruction, three chunks in flight (the load path's
//    full rate needs whole lines and this many bytes in flight); B past the
//    caches' retention (non-temporal), since it is read once.
//  * Within a chunk each wave multiplies one 32-row group of A by B over its
//    share of the chunk's 64-k steps, from zero: the share lies within one
//    group of 128 k, so the result times the two steps goes into the wave's
//    running sums.  The steps of a chunk (each row's and each column's, or
//    B's tile's, for its 4 groups) come into LDS with it, one load per wave.
//  * The waves' sums meet in LDS in a fixed order, take the bias and are
//    rounded once.

#include "block_gemm_tile.hpp"

namespace fp8lin {

namespace {

constexpr int kCols = 32;   // output columns per workgroup
constexpr int kWaves = 8;
constexpr int kChunk = 512;  // k per chunk: 4 groups, 8 matrix steps
constexpr int kGroups = kChunk / kGroup;
constexpr int kRing = 3;
constexpr int kRedStride = 36;  // floats per row of a partial tile in LDS

struct SkinnyParams {
    const uint8_t* a;
    const uint8_t* b;
    BlockScale sa, sb;
    const uint16_t* bias;
    uint16_t* out;
    int64_t m, n, k, lda, ldb;
    int xcd_remap;
};

__device__ __forceinline__ void dma16_nt(const v4i& rsrc, uint32_t lds, uint32_t voff) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds"
                 :
                 : "v"(voff), "s"(rsrc), "{m0}"(lds));
}

// MT: 32-row groups of A (1 when m <= 32, else 2).
template <int FA, int FB, int MT>
__global__ __launch_bounds__(kWaves * 64, 1) void block_gemm_skinny_kernel(SkinnyParams p) {
    // A chunk is [32 MT rows of A + 32 of B][512 B], the 16-byte pieces of
    // row r at index c ^ (r % 16); its steps [32 MT + 32 lines][4 groups].
    constexpr int kRowsA = 32 * MT, kRows = kRowsA + kCols;
    constexpr int kChunkBytes = kRows * kChunk;
    constexpr int kInstr = kRows / 2;  // 1 KB load instructions (2 rows) per chunk
    constexpr int kPer = kInstr / kWaves + 1;  // loads per wave, the steps' last
    constexpr int kSteps = kRows * kGroups, kStepsPer = kSteps / kWaves;
    static_assert(kInstr % kWaves == 0 && kSteps % kWaves == 0 && kStepsPer <= 64, "even shares");
    static_assert(kPer * (kRing - 1) < 64, "vmcnt range");
    constexpr int kRedBytes = (kWaves / MT) * kRowsA * kRedStride * 4;
    static_assert(kRedBytes <= kRing * kChunkBytes, "reduction fits the ring");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kRing * (kChunkBytes + 4 * kSteps)];
    uint8_t* steps = smem + kRing * kChunkBytes;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int bid = blockIdx.x;
    if (p.xcd_remap) bid = (bid & 7) * (gridDim.x >> 3) + (bid >> 3);
    const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(bid) * kCols;

    const int c4 = 4 * (threadIdx.x % (kCols / 4));  // epilogue columns of this thread
    float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p.bias) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (n0 + c4 + c < p.n) bias[c] = bf16_to_f32(p.bias[n0 + c4 + c]);
    }

    const v4i ra = make_rsrc(p.a);
    const v4i rb = make_rsrc(p.b + n0 * p.ldb);
    const int kdim = (int)p.k;
    const int nk = (kdim + kGroup - 1) / kGroup;

    // This lane's step: line and group within a chunk.  Lines past the matrix
    // and groups past k read the last one's.
    uint64_t step_at;
    uint32_t step_k;
    int step_g;
    {
        const int e = wave * kStepsPer + (lane < kStepsPer ? lane : 0);
        const int line = e / kGroups;
        step_g = e % kGroups;
        const bool is_b = line >= kRowsA;
        const int64_t lines = is_b ? p.n : p.m;
        int64_t i = is_b ? n0 + line - kRowsA : line;
        if (i >= lines) i = lines - 1;
        const BlockScale& s = is_b ? p.sb : p.sa;
        step_at = reinterpret_cast<uint64_t>(s.s + (i >> s.shift) * s.si);
        step_k = (uint32_t)(s.sk * 4);
    }

    const int half = lane >> 5, slot = lane & 31;
    auto issue = [&](int ring, int chunk) __attribute__((always_inline)) {
        const int k0 = chunk * kChunk;
        uint8_t* base = smem + ring * kChunkBytes;
#pragma unroll
        for (int j = 0; j < kPer - 1; ++j) {
            const int i = wave + j * kWaves;  // uniform
            const int row = 2 * i + half;
            const int kk = k0 + 16 * (slot ^ (row & 15));
            const bool is_a = 2 * i < kRowsA;  // uniform: both rows in A or in B
            const int r = is_a ? row : row - kRowsA;
            const bool ok = kk < kdim && (is_a ? r < p.m : n0 + r < p.n);
            const uint32_t off = ok ? (uint32_t)r * (uint32_t)(is_a ? p.lda : p.ldb) + kk : kOOB;
            if (is_a) dma16(ra, lds_addr(base + 1024 * i), off);
            else dma16_nt(rb, lds_addr(base + 1024 * i), off);
        }
        int g = chunk * kGroups + step_g;
        if (g >= nk) g = nk - 1;
        if (lane < kStepsPer)
            dma4(step_at + (uint64_t)g * step_k,
                 lds_addr(steps + 4 * (ring * kSteps + wave * kStepsPer)));
    };

    // Row group and share of a wave: MT consecutive 64-k steps of the chunk,
    // within group `grp_k` of it.
    constexpr int kParts = kWaves / MT;
    const int grp = wave % MT, part = wave / MT;
    const int grp_k = part * MT / 2;
    const int r32 = lane & 31;
    uint32_t flo[MT], fhi[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int c0 = 4 * (part * MT + j) + 2 * half;
        flo[j] = (uint32_t)(r32 * kChunk + 16 * (c0 ^ (r32 & 15)));
        fhi[j] = (uint32_t)(r32 * kChunk + 16 * ((c0 + 1) ^ (r32 & 15)));
    }
    auto frag = [&](const uint8_t* rows, int j) __attribute__((always_inline)) {
        const v4i x = *reinterpret_cast<const __attribute__((address_space(3))) v4i*>(
            (lds_void*)(rows + flo[j]));
        const v4i y = *reinterpret_cast<const __attribute__((address_space(3))) v4i*>(
            (lds_void*)(rows + fhi[j]));
        v8i v;
        v[0] = x[0]; v[1] = x[1]; v[2] = x[2]; v[3] = x[3];
        v[4] = y[0]; v[5] = y[1]; v[6] = y[2]; v[7] = y[3];
        return v;
    };
    auto barrier = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    typedef const __attribute__((address_space(3))) float lds_f32;
    auto step = [&](int ring, int line) __attribute__((always_inline)) {
        return *reinterpret_cast<lds_f32*>(
            (lds_void*)(steps + 4 * (ring * kSteps + line * kGroups + grp_k)));
    };

    // sum[e] is row 32 grp + lane % 32, column 8 (e / 4) + 4 (lane / 32) + e % 4
    v16f sum;
#pragma unroll
    for (int e = 0; e < 16; ++e) sum[e] = 0.0f;
    const int nch = (kdim + kChunk - 1) / kChunk;
#pragma unroll
    for (int c = 0; c < kRing; ++c)
        if (c < nch) issue(c, c);
    for (int c0 = 0; c0 < nch; c0 += kRing) {
#pragma unroll
        for (int q = 0; q < kRing; ++q) {
            const int c = c0 + q;
            if (c >= nch) break;
            const int ahead = nch - 1 - c;
            static_assert(kRing == 3, "wait cases");
            if (ahead >= 2) wait_vmcnt<2 * kPer>();
            else if (ahead == 1) wait_vmcnt<kPer>();
            else wait_vmcnt<0>();
            barrier();
            const uint8_t* base = smem + q * kChunkBytes;
            v8i fa[MT], fb[MT];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                fa[j] = frag(base + 32 * grp * kChunk, j);
                fb[j] = frag(base + kRowsA * kChunk, j);
            }
            const float sa = step(q, 32 * grp + r32);
            float sb[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) sb[e] = step(q, kRowsA + 8 * (e / 4) + 4 * half + e % 4);
            v16f pt = {0};
#pragma unroll
            for (int j = 0; j < MT; ++j) pt = mfma_ba<FA, FB>(fb[j], fa[j], pt);
            wait_lgkmcnt0();  // this slot is read before it is filled again
            barrier();
            if (c + kRing < nch) issue(q, c + kRing);
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[e] = fmaf(pt[e] * sa, sb[e], sum[e]);
        }
    }
    barrier();

    float* red = reinterpret_cast<float*>(smem);
    float* mine = red + part * (kRowsA * kRedStride);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v4f v;
        v[0] = sum[4 * q]; v[1] = sum[4 * q + 1]; v[2] = sum[4 * q + 2]; v[3] = sum[4 * q + 3];
        *reinterpret_cast<v4f*>(mine + (32 * grp + r32) * kRedStride + 8 * q + 4 * half) = v;
    }
    __syncthreads();
    constexpr int kOut = kRowsA * kCols / 4;  // 4-column groups of the tile
    for (int t = threadIdx.x; t < kOut; t += kWaves * 64) {
        const int row = t / (kCols / 4);
        if (row >= p.m) continue;
        v4f s = *reinterpret_cast<const v4f*>(red + row * kRedStride + c4);
#pragma unroll
        for (int w = 1; w < kParts; ++w)
            s += *reinterpret_cast<const v4f*>(red + w * (kRowsA * kRedStride) +
                                               row * kRedStride + c4);
        const int64_t gn = n0 + c4;
        const uint32_t w0 = f32x2_to_bf16x2(s[0] + bias[0], s[1] + bias[1]);
        const uint32_t w1 = f32x2_to_bf16x2(s[2] + bias[2], s[3] + bias[3]);
        uint16_t* dst = p.out + (int64_t)row * p.n + gn;
        if (gn + 3 < p.n && ((reinterpret_cast<uintptr_t>(dst) & 7) == 0)) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(w0, w1);
        } else {
            const uint16_t h[4] = {(uint16_t)w0, (uint16_t)(w0 >> 16), (uint16_t)w1,
                                   (uint16_t)(w1 >> 16)};
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (gn + c < p.n) dst[c] = h[c];
        }
    }
}

template <int FA, int FB>
void launch_formats(const SkinnyParams& p, dim3 grid, hipStream_t stream) {
    if (p.m <= 32)
        hipLaunchKernelGGL((block_gemm_skinny_kernel<FA, FB, 1>), grid, dim3(kWaves * 64), 0,
                           stream, p);
    else
        hipLaunchKernelGGL((block_gemm_skinny_kernel<FA, FB, 2>), grid, dim3(kWaves * 64), 0,
                           stream, p);
}

}  // namespace

hipError_t launch_block_skinny(const BlockGemmLaunch& g, hipStream_t stream) {
    SkinnyParams p{};
    p.a = g.a;
    p.b = g.b;
    p.sa = g.sa;
    p.sb = g.sb;
    p.bias = g.bias;
    p.out = g.out;
    p.m = g.m;
    p.n = g.n;
    p.k = g.k;
    p.lda = g.lda;
    p.ldb = g.ldb;
    const unsigned wgs = (unsigned)((g.n + kCols - 1) / kCols);
    p.xcd_remap = wgs % 8 == 0;
    if (g.fmt_a == 0) launch_formats<0, 0>(p, dim3(wgs), stream);
    else if (g.fmt_b == 0) launch_formats<1, 0>(p, dim3(wgs), stream);
    else launch_formats<1, 1>(p, dim3(wgs), stream);
    return hipGetLastError();
}

}  // namespace fp8lin
