// LDS-tiled block-scaled fp8 GEMM: the kernel template.  The instances are
// compiled per storage layout (block_gemm_{nt,nn,tn}.hip).
//
//   out[i][j] = bf16( sum_kb sa(i,kb) sb(kb,j) P_kb[i][j] + bias[j] ),
//   P_kb[i][j] = sum over the 128 k of group kb of A[i][k] B[k][j].
//
// The tiles, the ring of LDS stages and the operand layouts are the
// per-tensor kernel's (gemm_operand.hpp).  What is different:
//
//  * A stage holds 128 k: exactly one group.  Its two 64-k matrix
//    instructions start from zero and chain, so a 32 x 32 tile's P_kb is in 16
//    registers after them, and 16 fused multiply-adds put it, times the
//    steps, into the running sum.  Those take half the vector unit's time
//    that the two matrix instructions take of the matrix unit's, and run in
//    the shadow of the next tile's (the order below: in the second substep,
//    tile t - 1's sums follow tile t's matrix instruction; the last tile's
//    follow the next stage's first).
//  * The matrix instruction takes the B fragment first, so a lane's 16
//    values of a tile belong to one row of A: with one step per 128 x 128
//    tile of B the factor is one number per lane and tile.  With a step per
//    column (BVEC) each value has a factor of its own: twice the vector work,
//    and 16 registers more for every 32 columns of a wave, so that of the
//    three-stage tiles NT's 128 x 256 spills 15 registers and NN's two 2 and 3,
//    some of them read back inside the loop.
//  * The steps come into LDS with the operands.  Where both operands' lie
//    along k (A's rows, B's tiles) they come for ST stages at a time, with
//    the first of them (CHUNK): a row's next ones are in the same line, and
//    fetching it for each stage cost 4096^3 NT 4 us and 2048 x 1024 x 4096 NN
//    3.8 of 21.7.  Otherwise each stage brings its own, a line for every 32.

#pragma once

#include <type_traits>

#include "block.hpp"
#include "gemm_operand.hpp"

namespace fp8lin {

struct BlockTileParams {
    const uint8_t* a;
    const uint8_t* b;
    BlockScale sa, sb;
    const uint16_t* bias;
    uint16_t* out;
    int64_t m, n, k, lda, ldb;
    int tiles_m, tiles_n, group_m;
    int vec_out16;  // whole 16-byte chunks of output rows (and bias), aligned
    int xcd_remap;
    // Split along k: `splits` workgroups share a tile, each taking
    // groups_per groups; partial sums and a counter per tile in a workspace.
    int splits, groups_per;
    float* part;
    uint32_t* counters;
};

// One global -> LDS load of a dword per lane: lane l's goes to LDS at M0 + 4 l.
// No output register (see dma16).
__device__ __forceinline__ void dma4(uint64_t addr, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" : : "v"(addr), "{m0}"(lds));
}

// Keeps what is computed from x after this point and what x is computed from
// before it: the order of the matrix and vector instructions below is what
// bounds the registers, and nothing else would hold it.
__device__ __forceinline__ void pin(v8i& x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ void pin(float (&x)[16]) {
    asm volatile(""
                 : "+v"(x[0]), "+v"(x[1]), "+v"(x[2]), "+v"(x[3]), "+v"(x[4]), "+v"(x[5]),
                   "+v"(x[6]), "+v"(x[7]), "+v"(x[8]), "+v"(x[9]), "+v"(x[10]), "+v"(x[11]),
                   "+v"(x[12]), "+v"(x[13]), "+v"(x[14]), "+v"(x[15]));
}

template <class T>
__device__ __forceinline__ T* lds_at(uint32_t address) {
    return (T*)(uintptr_t)address;
}

// The same from a descriptor, 32-bit offset per lane and uniform offset.
__device__ __forceinline__ void dma4_at(const v4i& rsrc, uint32_t lds, uint32_t voff, int soff) {
    asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds));
}

template <int FA, int FB>
__device__ __forceinline__ v16f mfma_ba(const v8i& b, const v8i& a, v16f acc) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, FB, FA, 0, 0, 0, 0);
}

template <bool AMN, bool BVEC, int BM, int BN, int WM, int WN, int ST>
struct BlockTile {
    static constexpr int NW = WM * WN;
    static constexpr int kStage = (BM + BN) * kGroup;  // operand bytes of a stage
    static constexpr int kNB = BVEC ? BN : (BN + kGroup - 1) / kGroup;  // B's steps
    static constexpr bool CHUNK = !AMN && !BVEC && ST >= 3;
    // steps of a load (a stage, or ST of them), entries line * D + group
    static constexpr int D = CHUNK ? ST : 1;
    static constexpr int kEntries = (BM + kNB) * D;
    static constexpr int kPer = (kEntries + NW - 1) / NW;  // of each wave
    static constexpr int kStepLoads = (kPer + 63) / 64;    // a step per lane and load
    // floats per slot (the large tile's loop lays them out with room between)
    static constexpr int kSteps = (kPer * NW + 31) / 32 * 32 + (BM * BN == 256 * 256 ? 96 : 0);
    static constexpr int kStepSlots = CHUNK ? 2 : ST;
    static constexpr int kLds = ST * kStage + kStepSlots * 4 * kSteps;
    static_assert(kLds <= 160 * 1024, "LDS");
};

// One output tile: workgroup `bid` of a grid of `wgs` over problem p.  With
// SPLIT it is one share of a tile along k: the sums go to the workspace at
// device scope, and the workgroup that brings the last share adds them all, in
// the shares' order, and writes the tile.
template <int FA, int FB, bool AMN, bool BMN, bool BVEC, int BM, int BN, int WM, int WN, int ST,
          bool SPLIT = false>
__device__ __forceinline__ void block_gemm_tile(const BlockTileParams& p, int bid, int wgs,
                                                uint8_t* smem) {
    using BT = BlockTile<AMN, BVEC, BM, BN, WM, WN, ST>;
    constexpr int NW = BT::NW, BK = kGroup, kStage = BT::kStage, kPer = BT::kPer;
    constexpr int kStageA = BM * BK;
    constexpr int TM = BM / WM, TN = BN / WN;
    constexpr int FM = TM / 32, FN = TN / 32, kMF = FM * FN;
    // 128 x 64 per wave: partial sums and A's fragments of all its tiles do
    // not fit the registers beside the sums, so it goes row tile by row tile.
    constexpr bool BIG = FM == 4 && FN == 2;
    static_assert(!BIG || (ST == 2 && !BVEC), "the large tile's loop");
    static_assert(TN <= kGroup && kGroup % TN == 0, "a wave's columns share a tile of B");
    using OA = Operand<AMN, BM, NW, BK>;
    using OB = Operand<BMN, BN, NW, BK>;
    constexpr int kPA = OA::kPerWave, kPB = OB::kPerWave;
    // loads per wave and stage: operands, and steps with every stage or with
    // those of ring slot 0
    constexpr int kOps = kPA + kPB;
    constexpr int kStepLoads = BT::kStepLoads;
    constexpr bool CHUNK = BT::CHUNK;
    constexpr int kLoads = CHUNK ? kOps : kOps + kStepLoads;
    auto loads_of = [](int slot) constexpr { return CHUNK && slot == 0 ? kOps + kStepLoads : kLoads; };
    static_assert(ST >= 2 && kLoads * (ST - 1) + kStepLoads < 64, "vmcnt range");
    uint8_t* steps = smem + ST * kStage;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    if (p.xcd_remap) bid = (bid & 7) * (wgs >> 3) + (bid >> 3);
    int share = 0;
    if constexpr (SPLIT) {
        const int tiles = p.tiles_m * p.tiles_n;
        share = bid / tiles;
        bid -= share * tiles;
    }
    const int per_group = p.group_m * p.tiles_n;
    const int first_m = (bid / per_group) * p.group_m;
    const int gsz = p.tiles_m - first_m < p.group_m ? p.tiles_m - first_m : p.group_m;
    const int r = bid - (bid / per_group) * per_group;
    const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane((first_m + r % gsz) * BM);
    const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane((r / gsz) * BN);

    const int g0 = SPLIT ? share * p.groups_per : 0;  // first group of k
    const int64_t k0 = (int64_t)g0 * BK;
    const v4i ra = make_rsrc(p.a + (AMN ? m0 + k0 * p.lda : m0 * p.lda + k0));
    const v4i rb = make_rsrc(p.b + (BMN ? n0 + k0 * p.ldb : n0 * p.ldb + k0));
    const uint32_t lda = (uint32_t)p.lda, ldb = (uint32_t)p.ldb;
    const int left = (int)(p.k - k0);
    const int kdim = SPLIT && left > p.groups_per * BK ? p.groups_per * BK : left;
    const int nk = (kdim + BK - 1) / BK;
    const int64_t arows = p.m - m0, brows = p.n - n0;
    const bool afull = arows >= BM, bfull = brows >= BN;
    const uint32_t abase = OA::init(lda, arows, wave, lane);
    const uint32_t bbase = OB::init(ldb, brows, wave, lane);

    // This lane's steps: address at group 0 (with CHUNK, at its group of a
    // chunk) and the bytes to the next group.  Lines past the matrix read its
    // last one's.
    uint64_t step_at[kStepLoads];
    uint32_t step_k[kStepLoads];
    int step_g[kStepLoads];
#pragma unroll
    for (int x = 0; x < kStepLoads; ++x) {
        const int in = 64 * x + lane < kPer ? 64 * x + lane : kPer - 1;
        int e = wave * kPer + in;
        if (e >= BT::kEntries) e = BT::kEntries - 1;
        const int line = e / BT::D;
        step_g[x] = e % BT::D;
        const bool is_b = line >= BM;
        int64_t i;
        if (!is_b) {
            i = m0 + line < p.m ? m0 + line : p.m - 1;
        } else {
            const int64_t j = BVEC ? n0 + (line - BM) : (n0 / kGroup + (line - BM)) * kGroup;
            i = j < p.n ? j : p.n - 1;
        }
        const BlockScale& s = is_b ? p.sb : p.sa;
        step_at[x] = reinterpret_cast<uint64_t>(s.s + (i >> s.shift) * s.si + g0 * s.sk);
        step_k[x] = (uint32_t)(s.sk * 4);
    }
    // Load x of the stage at group kg into ring slot s.
    auto load = [&](int x, int s, int kg) __attribute__((always_inline)) {
        uint8_t* dst = smem + s * kStage;
        if (x < kPA) {
            dma16(ra, OA::lds_of(dst, x, wave),
                  OA::off_of(abase, lda, kg * BK, kdim, afull, arows, x, wave, lane));
        } else if (x < kPA + kPB) {
            dma16(rb, OB::lds_of(dst + kStageA, x - kPA, wave),
                  OB::off_of(bbase, ldb, kg * BK, kdim, bfull, brows, x - kPA, wave, lane));
        } else {
            const int y = x - kPA - kPB;
            const int slot = CHUNK ? kg / ST & 1 : s;
            int g = kg + step_g[y];
            if (g >= nk) g = nk - 1;  // past the end: any group
            if (64 * y + lane < kPer)
                dma4(step_at[y] + (uint64_t)g * step_k[y],
                     lds_addr(steps + 4 * (slot * BT::kSteps + wave * kPer + 64 * y)));
        }
    };

    v8i af[2][BIG ? 1 : FM], bf[2][FN];
    uint32_t aoff[FM], boff[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) aoff[i] = OA::frag_off(AMN ? wm * TM + 32 * i : 0, lane);
#pragma unroll
    for (int j = 0; j < FN; ++j) boff[j] = OB::frag_off(BMN ? wn * TN + 32 * j : 0, lane);
    constexpr int kRowA = AMN ? 0 : BK, kRowB = BMN ? 0 : BK;
    const uint32_t arow = (uint32_t)(wm * TM * kRowA), brow = (uint32_t)(wn * TN * kRowB);

    auto barrier = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    constexpr int kParts = BIG ? FN : kMF;
    // (the sums are plain numbers: only `part` is a matrix register tuple)
    float acc[FM][FN][16];
    v16f part[kParts];
#pragma unroll
    for (int t = 0; t < kMF; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[t % FM][t / FM][e] = 0.0f, part[t % kParts][e] = 0.0f;
    // The steps of the stage in work: rows', and with BVEC columns' (16 of
    // each 32-column tile); prev_a: the last tile's of the stage before.
    // With BVEC the last tile is summed in its own stage: carrying its
    // columns' steps over would cost 16 registers that there are not.
    float sa[FM], prev_a = 0.0f;
    v4f sb[BVEC ? FN : 1][4];
    typedef const __attribute__((address_space(3))) float lds_f32;
    typedef const __attribute__((address_space(3))) v4f lds_v4f;
    // ring slot s of the turn `turn` of the ring
    auto read_steps = [&](int s, int turn) __attribute__((always_inline)) {
        uint8_t* at = steps + 4 * (CHUNK ? (turn & 1) * BT::kSteps + s : s * BT::kSteps);
        if constexpr (BVEC) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sb[j][q] = *reinterpret_cast<lds_v4f*>(
                        (lds_void*)(at + 4 * (BM + wn * TN + 32 * j + 8 * q + 4 * (lane >> 5))));
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
            sa[i] = *reinterpret_cast<lds_f32*>(
                (lds_void*)(at + 4 * BT::D * (wm * TM + 32 * i + (lane & 31))));
        if constexpr (!BVEC) {
            const float b = *reinterpret_cast<lds_f32*>(
                (lds_void*)(at + 4 * BT::D * (BM + wn * TN / kGroup)));
#pragma unroll
            for (int i = 0; i < FM; ++i) sa[i] *= b;
        }
    };
    auto fold = [&](float (&a)[16], const v16f& pt, float fa, const v4f* fb)
                    __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if constexpr (BVEC) a[e] = fmaf(pt[e] * fa, fb[e / 4][e % 4], a[e]);
            else a[e] = fmaf(pt[e], fa, a[e]);
        }
    };

    if constexpr (BIG) {
        // Per row tile i: two matrix instructions of each column tile on the
        // first 64 k, then two on the second, and behind them the sums:
        //   M(0,j0)  sum(i-1,j1)  M(0,j1)  M(1,j0)  M(1,j1)  sum(i,j0)
        // A's fragments of the next row tile replace each half's as soon as
        // it is used.  The stage ends inside its last row tile: once the
        // first half's instructions are out, nothing of the slot is left to
        // read but what has arrived, so the barrier comes there, and the
        // second half's instructions cover the next stage's first reads.
        //
        // 128 sums, 32 partial ones and 48 fragment registers leave about 40
        // for all else, and a register spilled inside the loop would be read
        // back behind every load in flight (NT keeps one in memory, stored before
        // the loop and read after it; NN and TN none): so the fragments' LDS addresses
        // are kept per slot and moved to the other one each stage, and the
        // steps come by 32-bit offsets from descriptors.
        typedef const __attribute__((address_space(3))) v4i lds_v4i;
        typedef __attribute__((address_space(3))) v2i lds_v2i;
        constexpr int kAddrA = AMN ? FM : 4, kAddrB = BMN ? FN : 4;
        uint32_t fa[kAddrA], fb[kAddrB];
#pragma unroll
        for (int x = 0; x < kAddrA; ++x)
            fa[x] = lds_addr(smem) + arow +
                    (AMN ? aoff[AMN ? x : 0] : aoff[0] ^ (64u * (x / 2) + 16u * (x % 2)));
#pragma unroll
        for (int x = 0; x < kAddrB; ++x)
            fb[x] = lds_addr(smem) + kStageA + brow +
                    (BMN ? boff[BMN ? x : 0] : boff[0] ^ (64u * (x / 2) + 16u * (x % 2)));
        auto frag = [&](auto mnc, auto rc, auto hc, const uint32_t* f, int i)
                        __attribute__((always_inline)) {
            constexpr int R = decltype(rc)::value, H = decltype(hc)::value;
            v8i v;
            if constexpr (!decltype(mnc)::value) {
                const v4i lo = *lds_at<lds_v4i>(f[2 * H] + 32 * i * BK);
                const v4i hi = *lds_at<lds_v4i>(f[2 * H + 1] + 32 * i * BK);
                v[0] = lo[0]; v[1] = lo[1]; v[2] = lo[2]; v[3] = lo[3];
                v[4] = hi[0]; v[5] = hi[1]; v[6] = hi[2]; v[7] = hi[3];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const v2i t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        lds_at<lds_v2i>(f[i] + (kSub * H + 8 * q) * R));
                    v[2 * q] = t[0];
                    v[2 * q + 1] = t[1];
                }
            }
            return v;
        };
        using TA = std::integral_constant<bool, AMN>;
        using TB = std::integral_constant<bool, BMN>;
        using RA = std::integral_constant<int, BM>;
        using RB = std::integral_constant<int, BN>;
        using I0 = std::integral_constant<int, 0>;
        using I1 = std::integral_constant<int, 1>;
        auto read_a = [&](auto hc, int i) __attribute__((always_inline)) {
            af[decltype(hc)::value][0] = frag(TA{}, RA{}, hc, fa, i);
        };
        auto read_b = [&](auto hc) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < FN; ++j) bf[decltype(hc)::value][j] = frag(TB{}, RB{}, hc, fb, j);
        };
        // Steps: rows 32 wave .. + 63 (half of them the next wave's too), and
        // by every wave the two of B's tiles, in all 64 lanes: the same values
        // meet in the same places, and no lane has to be masked.
        const v4i rsa = make_rsrc(p.sa.s + g0 * p.sa.sk), rsb = make_rsrc(p.sb.s + g0 * p.sb.sk);
        const int ska = (int)p.sa.sk * 4, skb = (int)p.sb.sk * 4;
        uint32_t voa, vob;
        {
            const int64_t i = m0 + 32 * wave + lane, j = n0 + (lane & 1) * kGroup;
            voa = (uint32_t)(((i < p.m ? i : p.m - 1) >> p.sa.shift) * p.sa.si * 4);
            vob = (uint32_t)(((j < p.n ? j : p.n - 1) >> p.sb.shift) * p.sb.si * 4);
        }
        constexpr int kStepB = BM + 32, kStepRow = kStepB + 64;  // floats per slot
        static_assert(2 * kStepRow <= ST * BT::kSteps, "the slots fit");
        const uint32_t steps_at = lds_addr(steps);
        constexpr int kBigLoads = kPA + kPB + 2;
        // load x of the stage at group kg into slot s
        auto big_load = [&](int x, int s, int kg) __attribute__((always_inline)) {
            if (x < kPA + kPB) {
                load(x, s, kg);
            } else {
                const int g = kg < nk ? kg : nk - 1;
                const uint32_t at = steps_at + 4 * s * kStepRow;
                if (x == kPA + kPB) dma4_at(rsa, at + 128 * wave, voa, g * ska);
                else dma4_at(rsb, at + 4 * kStepB, vob, g * skb);
            }
        };
        auto big_steps = [&](int s) __attribute__((always_inline)) {
            const uint32_t at = steps_at + 4 * s * kStepRow;
            const float b = *lds_at<lds_f32>(at + 4 * (kStepB + wn * TN / kGroup));
#pragma unroll
            for (int i = 0; i < FM; ++i)
                sa[i] = *lds_at<lds_f32>(at + 4 * (wm * TM + 32 * i + (lane & 31))) * b;
        };
#pragma unroll
        for (int x = 0; x < kBigLoads; ++x) big_load(x, 0, 0);
#pragma unroll
        for (int x = 0; x < 2; ++x) big_load(x, 1, 1);
        wait_vmcnt<2>();
        barrier();
        read_a(I0{}, 0);
        read_b(I0{});
        read_a(I1{}, 0);
        read_b(I1{});
        big_steps(0);
        const v16f zero = {0};
        int move = kStage;  // to the other slot
        for (int st = 0, s = 0; st < nk; ++st, s ^= 1) {
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                pin(af[0][0]);
                part[0] = mfma_ba<FA, FB>(bf[0][0], af[0][0], zero);
                // the row tile before's second sums
                fold(acc[(i + FM - 1) % FM][1], part[1], i == 0 ? prev_a : sa[(i + FM - 1) % FM],
                     nullptr);
                pin(acc[(i + FM - 1) % FM][1]);
                __builtin_amdgcn_sched_barrier(0);
                pin(af[0][0]);
                part[1] = mfma_ba<FA, FB>(bf[0][1], af[0][0], zero);
                if (i + 1 < FM) {
                    read_a(I0{}, i + 1);
                    // the rest of the refill that the stage before began
                    constexpr int kPerTile = (kBigLoads - 2 + 1) / 2;
                    if (i < 2) {
#pragma unroll
                        for (int x = 2 + i * kPerTile; x < 2 + (i + 1) * kPerTile; ++x)
                            if (x < kBigLoads) big_load(x, s ^ 1, st + 1);
                    }
                } else {
                    wait_vmcnt<0>();  // this wave's loads of stage st + 1
                    wait_lgkmcnt0();  // and its reads of this stage
                    barrier();
#pragma unroll
                    for (int x = 0; x < kAddrA; ++x) fa[x] += move;
#pragma unroll
                    for (int x = 0; x < kAddrB; ++x) fb[x] += move;
                    move = -move;
                    read_a(I0{}, 0);
                    read_b(I0{});
                }
                __builtin_amdgcn_sched_barrier(0);
                pin(af[1][0]);
                part[0] = mfma_ba<FA, FB>(bf[1][0], af[1][0], part[0]);
                __builtin_amdgcn_sched_barrier(0);
                pin(af[1][0]);
                part[1] = mfma_ba<FA, FB>(bf[1][1], af[1][0], part[1]);
                if (i + 1 < FM) {
                    read_a(I1{}, i + 1);
                } else {
                    read_a(I1{}, 0);
                    read_b(I1{});
#pragma unroll
                    for (int x = 0; x < 2; ++x) big_load(x, s, st + ST);
                }
                fold(acc[i][0], part[0], sa[i], nullptr);
                pin(acc[i][0]);
                __builtin_amdgcn_sched_barrier(0);
            }
            prev_a = sa[FM - 1];
            big_steps(s ^ 1);
        }
    } else {
        // Substep H of the stage in slot s: its matrix instructions; between
        // them the reads of the next substep's fragments (slot ns) and loads
        // [X0, X1) of the refill of slot rs with group rk.
        constexpr int kFR = FM + FN, kFRPer = (kFR + kMF - 1) / kMF;
        auto substep = [&](auto hc, int ns, auto x0c, auto x1c, int rs, int rk)
                           __attribute__((always_inline)) {
            constexpr int H = decltype(hc)::value;
            constexpr int X0 = decltype(x0c)::value, X1 = decltype(x1c)::value;
            constexpr int kDPer = (X1 - X0 + kMF - 1) / kMF;
            const uint8_t* la = smem + ns * kStage + arow;
            const uint8_t* lb = smem + ns * kStage + kStageA + brow;
#pragma unroll
            for (int t = 0; t < kMF; ++t) {
                const int i = t % FM, j = t / FM;
                if constexpr (H == 0) {
                    const v16f zero = {0};
                    // (with one tile per wave its registers are needed at once)
                    if (!BVEC && kMF == 1) fold(acc[0][0], part[0], prev_a, nullptr);
                    part[t] = mfma_ba<FA, FB>(bf[0][j], af[0][i], zero);
                    if (!BVEC && kMF > 1 && t == 0)
                        fold(acc[FM - 1][FN - 1], part[kMF - 1], prev_a, nullptr);
                } else {
                    part[t] = mfma_ba<FA, FB>(bf[1][j], af[1][i], part[t]);
                    if (t > 0) {
                        const int u = t - 1;
                        fold(acc[u % FM][u / FM], part[u], sa[u % FM], sb[BVEC ? u / FM : 0]);
                    }
                }
#pragma unroll
                for (int q = 0; q < kFRPer; ++q) {
                    const int x = t * kFRPer + q;
                    if (x < FM) af[1 - H][x] = OA::template frag<1 - H>(la + 32 * x * kRowA, aoff[x]);
                    else if (x < kFR)
                        bf[1 - H][x - FM] =
                            OB::template frag<1 - H>(lb + 32 * (x - FM) * kRowB, boff[x - FM]);
                }
#pragma unroll
                for (int q = 0; q < kDPer; ++q) {
                    const int x = X0 + t * kDPer + q;
                    if (x < X1) load(x, rs, rk);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (H == 1) {
                if constexpr (BVEC) fold(acc[FM - 1][FN - 1], part[kMF - 1], sa[FM - 1], sb[FN - 1]);
                else prev_a = sa[FM - 1];
            }
        };
        // A refill's loads go out over two substeps when the ring has the slack
        // (three stages or more): the first kH after the barrier that frees the
        // slot, the rest in the next stage's first substep.
        constexpr bool kSplit = ST >= 3;
        constexpr int kH = kSplit ? (kLoads + 1) / 2 : kLoads;
        static_assert(kSplit || !CHUNK, "the steps go with a refill's second part");
        using I0 = std::integral_constant<int, 0>;
        using I1 = std::integral_constant<int, 1>;
        using IH = std::integral_constant<int, kH>;
        using IL = std::integral_constant<int, kLoads>;
        using IL0 = std::integral_constant<int, loads_of(0)>;

#pragma unroll
        for (int s = 0; s < ST - 1; ++s)
#pragma unroll
            for (int x = 0; x < loads_of(s); ++x) load(x, s, s);
#pragma unroll
        for (int x = 0; x < kH; ++x) load(x, ST - 1, ST - 1);
        wait_vmcnt<kLoads * (ST - 2) + kH>();
        barrier();
#pragma unroll
        for (int i = 0; i < FM; ++i) af[0][i] = OA::template frag<0>(smem + arow + 32 * i * kRowA, aoff[i]);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            bf[0][j] = OB::template frag<0>(smem + kStageA + brow + 32 * j * kRowB, boff[j]);

        for (int t0 = 0, turn = 0; t0 < nk; t0 += ST, ++turn) {
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                const int st = t0 + s;
                if (st >= nk) break;
                read_steps(s, turn);
                // the rest of the refill that stage st - 1 began
                const int prev = (s + ST - 1) % ST;
                if (prev == 0) substep(I0{}, s, IH{}, IL0{}, prev, st + ST - 1);
                else substep(I0{}, s, IH{}, IL{}, prev, st + ST - 1);
                // This wave's loads of stage st + 1 (what may be out are those of
                // the ST - 2 after it, slot 0's steps among them or not), and its
                // reads of this stage.
                if (CHUNK && s >= 1 && s <= ST - 2) wait_vmcnt<kLoads * (ST - 2) + kStepLoads>();
                else wait_vmcnt<kLoads * (ST - 2)>();
                wait_lgkmcnt0();
                barrier();
                substep(I1{}, (s + 1) % ST, I0{}, IH{}, s, st + ST);
            }
        }
    }
    if constexpr (!BVEC) fold(acc[FM - 1][FN - 1], part[kParts - 1], prev_a, nullptr);
    wait_vmcnt<0>();  // the prefetches past the end

    if constexpr (SPLIT) {
        // a lane's sums as pairs: pair q of lane l of a tile is 64 q + l
        const int tiles = p.tiles_m * p.tiles_n;
        auto at = [&](int sh, int t) {
            return reinterpret_cast<uint64_t*>(p.part) +
                   (((int64_t)sh * tiles + bid) * NW + wave) * (kMF * 512) + t * 512 + lane;
        };
#pragma unroll
        for (int t = 0; t < kMF; ++t)
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float(&v)[16] = acc[t % FM][t / FM];
                const uint64_t pair = __float_as_uint(v[2 * q]) |
                                      (uint64_t)__float_as_uint(v[2 * q + 1]) << 32;
                __hip_atomic_store(at(share, t) + 64 * q, pair, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            }
        wait_vmcnt<0>();  // the stores have reached device scope
        barrier();
        if (tid == 0) {
            const uint32_t seen = __hip_atomic_fetch_add(p.counters + bid, 1u, __ATOMIC_RELAXED,
                                                         __HIP_MEMORY_SCOPE_AGENT);
            if (seen == (uint32_t)p.splits - 1)
                __hip_atomic_store(p.counters + bid, 0u, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            *reinterpret_cast<uint32_t*>(smem) = seen == (uint32_t)p.splits - 1;
        }
        __syncthreads();
        if (*reinterpret_cast<volatile uint32_t*>(smem) == 0) return;
#pragma unroll
        for (int t = 0; t < kMF; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[t % FM][t / FM][e] = 0.0f;
        // four shares' loads at a time: each takes about a microsecond
        constexpr int kAhead = 4;
        for (int s0 = 0; s0 < p.splits; s0 += kAhead)
#pragma unroll
            for (int t = 0; t < kMF; ++t) {
                uint64_t pair[kAhead][8];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        pair[i][q] = __hip_atomic_load(
                            at(s0 + i < p.splits ? s0 + i : s0, t) + 64 * q, __ATOMIC_RELAXED,
                            __HIP_MEMORY_SCOPE_AGENT);
                float(&v)[16] = acc[t % FM][t / FM];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (s0 + i >= p.splits) break;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        v[2 * q] += __uint_as_float((uint32_t)pair[i][q]);
                        v[2 * q + 1] += __uint_as_float((uint32_t)(pair[i][q] >> 32));
                    }
                }
            }
        barrier();  // the flag is read before the tile is staged over it
    }

    // acc[i][j][e] is row m0 + wm*TM + 32i + lane%32, column
    // n0 + wn*TN + 32j + 8*(e/4) + 4*(lane/32) + e%4: through LDS, as the
    // per-tensor kernel, so that the stores go by rows (in 16-byte chunks,
    // swizzled by row, where the output's rows are whole ones).
    constexpr int kRowBytes = TN * 2, kChunks = kRowBytes / 16;
    constexpr int kRowsPerPass = 64 / kChunks, kRegion = TM * kRowBytes;
    static_assert(NW * kRegion <= ST * kStage, "epilogue staging fits the ring");
    barrier();
    uint8_t* wl = smem + wave * kRegion;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int cl = 32 * j + 8 * q + 4 * (lane >> 5);
            const int64_t gn = n0 + wn * TN + cl;
            float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (p.bias) {
                if (p.vec_out16) {
                    if (gn < p.n) {
                        const uint2 bb = *reinterpret_cast<const uint2*>(p.bias + gn);
                        bias[0] = bf16_lo(bb.x); bias[1] = bf16_hi(bb.x);
                        bias[2] = bf16_lo(bb.y); bias[3] = bf16_hi(bb.y);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (gn + c < p.n) bias[c] = bf16_to_f32(p.bias[gn + c]);
                }
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int row = 32 * i + (lane & 31);
                const int chunk = (cl >> 3) ^ (row % kChunks);
                v2i pk;
                pk[0] = (int)f32x2_to_bf16x2(acc[i][j][4 * q + 0] + bias[0],
                                             acc[i][j][4 * q + 1] + bias[1]);
                pk[1] = (int)f32x2_to_bf16x2(acc[i][j][4 * q + 2] + bias[2],
                                             acc[i][j][4 * q + 3] + bias[3]);
                *reinterpret_cast<__attribute__((address_space(3))) v2i*>(
                    (lds_void*)(wl + row * kRowBytes + chunk * 16 + 8 * (lane >> 5))) = pk;
            }
        }
    }
    if (p.vec_out16) {
        const int cc = lane % kChunks;
        const int64_t gn = n0 + wn * TN + 8 * cc;
#pragma unroll
        for (int ps = 0; ps < TM / kRowsPerPass; ++ps) {
            const int row = ps * kRowsPerPass + lane / kChunks;
            const v4i v = *reinterpret_cast<const __attribute__((address_space(3))) v4i*>(
                (lds_void*)(wl + row * kRowBytes + ((cc ^ (row % kChunks)) << 4)));
            const int64_t gm = m0 + wm * TM + row;
            if (gm < p.m && gn < p.n) *reinterpret_cast<v4i*>(p.out + gm * p.n + gn) = v;
        }
        return;
    }
    constexpr int kRowsPer = 64 / TN;  // one output a lane
    static_assert(TN <= 64, "a lane per column");
    const int col = lane % TN;
    const int64_t gn = n0 + wn * TN + col;
    for (int ps = 0; ps < TM / kRowsPer; ++ps) {
        const int row = ps * kRowsPer + lane / TN;
        const int64_t gm = m0 + wm * TM + row;
        const uint16_t v = *reinterpret_cast<const __attribute__((address_space(3))) uint16_t*>(
            (lds_void*)(wl + row * kRowBytes + (((col >> 3) ^ (row % kChunks)) << 4) +
                        2 * (col & 7)));
        if (gm < p.m && gn < p.n) p.out[gm * p.n + gn] = v;
    }
}

template <int FA, int FB, bool AMN, bool BMN, bool BVEC, int BM, int BN, int WM, int WN, int ST>
__global__ __launch_bounds__(WM* WN * 64, 1) void block_gemm_kernel(BlockTileParams p) {
    __shared__ __attribute__((aligned(1024)))
    uint8_t smem[BlockTile<AMN, BVEC, BM, BN, WM, WN, ST>::kLds];
    block_gemm_tile<FA, FB, AMN, BMN, BVEC, BM, BN, WM, WN, ST>(p, blockIdx.x, gridDim.x, smem);
}

template <int FA, int FB, bool AMN, bool BMN, bool BVEC, int BM, int BN, int WM, int WN, int ST>
__global__ __launch_bounds__(WM* WN * 64, 1) void block_gemm_split_kernel(BlockTileParams p) {
    __shared__ __attribute__((aligned(1024)))
    uint8_t smem[BlockTile<AMN, BVEC, BM, BN, WM, WN, ST>::kLds];
    block_gemm_tile<FA, FB, AMN, BMN, BVEC, BM, BN, WM, WN, ST, true>(p, blockIdx.x, gridDim.x,
                                                                     smem);
}

// Tiles: kWide 128 x 256, kTall 256 x 128, kMid 128 x 128, kSmall 64 x 64,
// kBig 256 x 256 (a step per tile of B).
enum class BlockCfg { kWide, kTall, kMid, kSmall, kBig };
// How a product of 64 x 64 tiles is split along k: 1 for not at all.
int block_gemm_splits(int64_t m, int64_t n, int64_t k);
hipError_t launch_block_skinny(const BlockGemmLaunch& g, hipStream_t stream);  // NT, m <= 64
hipError_t launch_block_nt(const BlockGemmLaunch& g, bool bvec, BlockCfg c, hipStream_t stream);
hipError_t launch_block_nn(const BlockGemmLaunch& g, bool bvec, BlockCfg c, hipStream_t stream);
hipError_t launch_block_tn(const BlockGemmLaunch& g, bool bvec, BlockCfg c, hipStream_t stream);

template <int BM, int BN>
BlockTileParams block_tile_params(const BlockGemmLaunch& g) {
    BlockTileParams p{};
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
    p.tiles_m = (int)((g.m + BM - 1) / BM);
    p.tiles_n = (int)((g.n + BN - 1) / BN);
    p.group_m = 4;
    const uintptr_t ob = reinterpret_cast<uintptr_t>(g.out);
    const uintptr_t bb = reinterpret_cast<uintptr_t>(g.bias);
    p.vec_out16 = (ob & 15) == 0 && g.n % 8 == 0 && (bb & 7) == 0;
    p.xcd_remap = p.tiles_m * p.tiles_n % 8 == 0;
    return p;
}

template <int FA, int FB, bool AMN, bool BMN, bool BVEC, int BM, int BN, int WM, int WN, int ST>
hipError_t launch_block_tile(const BlockGemmLaunch& g, hipStream_t stream) {
    const BlockTileParams p = block_tile_params<BM, BN>(g);
    hipLaunchKernelGGL((block_gemm_kernel<FA, FB, AMN, BMN, BVEC, BM, BN, WM, WN, ST>),
                       dim3((unsigned)(p.tiles_m * p.tiles_n)), dim3(WM * WN * 64), 0, stream, p);
    return hipGetLastError();
}

template <int FA, int FB, bool AMN, bool BMN, bool BVEC>
hipError_t launch_block_small(const BlockGemmLaunch& g, hipStream_t stream) {
    const int splits = g.part ? block_gemm_splits(g.m, g.n, g.k) : 1;
    if (splits == 1) return launch_block_tile<FA, FB, AMN, BMN, BVEC, 64, 64, 2, 2, 4>(g, stream);
    BlockTileParams p = block_tile_params<64, 64>(g);
    const int tiles = p.tiles_m * p.tiles_n;
    p.splits = splits;
    p.groups_per = (int)((groups_of(g.k) + splits - 1) / splits);
    p.part = g.part;
    p.counters = g.counters;
    p.xcd_remap = tiles * splits % 8 == 0;
    hipLaunchKernelGGL((block_gemm_split_kernel<FA, FB, AMN, BMN, BVEC, 64, 64, 2, 2, 4>),
                       dim3((unsigned)(tiles * splits)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

template <int FA, int FB, bool AMN, bool BMN, bool BVEC>
hipError_t launch_block_cfg(const BlockGemmLaunch& g, BlockCfg c, hipStream_t stream) {
    switch (c) {
        case BlockCfg::kBig:
            if constexpr (!BVEC)
                return launch_block_tile<FA, FB, AMN, BMN, BVEC, 256, 256, 2, 4, 2>(g, stream);
            else return hipErrorInvalidValue;  // (not chosen)
        case BlockCfg::kSmall: return launch_block_small<FA, FB, AMN, BMN, BVEC>(g, stream);
        case BlockCfg::kWide:
            return launch_block_tile<FA, FB, AMN, BMN, BVEC, 128, 256, 2, 4, 3>(g, stream);
        case BlockCfg::kTall:
            return launch_block_tile<FA, FB, AMN, BMN, BVEC, 256, 128, 4, 2, 3>(g, stream);
        default: break;
    }
    return launch_block_tile<FA, FB, AMN, BMN, BVEC, 128, 128, 4, 2, 4>(g, stream);
}

// Formats of one layout's instances: equal ones, and an E5M2 first operand
// with an E4M3 second (a gradient times what the forward quantized).
template <bool AMN, bool BMN>
hipError_t launch_block_layout(const BlockGemmLaunch& g, bool bvec, BlockCfg c,
                               hipStream_t stream) {
    auto pick = [&](auto bv) {
        constexpr bool V = decltype(bv)::value;
        if (g.fmt_a == 0) return launch_block_cfg<0, 0, AMN, BMN, V>(g, c, stream);
        return g.fmt_b == 0 ? launch_block_cfg<1, 0, AMN, BMN, V>(g, c, stream)
                            : launch_block_cfg<1, 1, AMN, BMN, V>(g, c, stream);
    };
    return bvec ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace fp8lin
