// Mixture-of-experts layer for a few tokens on tile-scaled fp8 weights:
//   l = x R^T;  the top_k experts e_j of each token (ties: lowest index);
//   w = softmax(l)[e_j], over their sum when asked;
//   y = sum_j w_j W2_e ( silu(G_e x) * (U_e x) ),  every weight = code * step.
//
// With few tokens per expert the layer is bound by reading the chosen
// experts' weights once (3 dim hidden bytes each), so both products are
// shaped for that.  (An expert's weights are read once for every 16 of its
// tokens: 8 experts of 2048 x 1024, 2 a token, 256 tokens take 93 us and 1024
// take 292.)
//
//  * The routing launch leaves a list of the experts that were reached and
//    of each one's tokens, so that a workgroup of the products knows its work
//    from one short read.  One token has a form of its own, whose workgroups
//    choose for themselves and add up the choices' shares in LDS.
//  * A workgroup takes 32 hidden units of one expert (32 rows of G and of U)
//    or 64 rows of W2, for all of the expert's tokens; its 4 waves take the
//    128-k blocks in turn, so every byte of x and of the weights is loaded by
//    one wave of it, and the four partial sums meet in LDS in a fixed order.
//  * Weights go straight into registers by whole lines, are brought into the
//    matrix instruction's layout by lane permutes, widened to bf16
//    (exact) and multiplied by bf16 activations: 16 tokens ride on one 16x16x32
//    instruction, so one token costs what 16 do.
//  * A block of 128 k lies in one tile of steps: its four instructions start
//    from zero, and the sum times the step is added in fp32.
//  * The hidden activations go between the two kernels as two bf16 numbers
//    each (the value rounded, and the rest rounded): 16 bits of precision
//    for one more matrix instruction, which the loads hide.

#include <type_traits>

#include "block.hpp"
#include "common.hpp"

namespace fp8lin {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxExperts = 512, kMaxTokens = 1024, kMaxTopK = 16;
constexpr int kRouteTokens = 4;   // tokens of a routing workgroup
constexpr int kTiles = 4;         // 16-row tiles of weights per wave
constexpr int kUnits = 8 * kTiles;        // hidden units of a gate / up workgroup
constexpr int kRows = 16 * kTiles;        // rows of W2 of a down workgroup
// From this many workgroups of a product on, a wave loads a block when it has
// used the one before, and its registers leave room for twice the waves on a
// CU; below it a wave loads one block ahead of the one that it multiplies.
// 64 experts of 2048 x 1024, 8 a token, whole layer: 64 tokens (2048
// workgroups) 100 us, 108 with one ahead; one token (256 workgroups; before it
// had its own form) 26.5 us, 25.7.
constexpr unsigned kManyGroups = 1024;

// One token: waves and outputs of a down workgroup (16 outputs a workgroup: 64
// experts of 2048 x 1024, 8 a token, 23.3 us instead of 22.4).
constexpr int kOneWaves = 8, kOneRows = 8;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// An expert that some token chose: its slots (token * top_k + rank) are
// slots[first .. first + count), in no particular order (each is a column of
// its own in the products).
struct Reached {
    int expert, first, count, pad;
};

// Workspace: counters first (zero between calls), then what one kernel
// leaves for the next.
struct MoeWs {
    uint32_t* route_count;  // per token group: routing workgroups done
    uint32_t* group_count;  // token groups done
    uint32_t* down_count;   // per kRows of the output and token: experts done
    int32_t* reached_n;     // experts reached
    Reached* reached;       // [min(experts, tokens * top_k)]
    int32_t* slots;         // [tokens * top_k]
    float* logits;          // [tokens][experts]
    int32_t* ids;           // [tokens][top_k]
    float* weights;         // [tokens][top_k]
    uint16_t* h;            // bf16 [tokens * top_k][moe_h_row(hidden)]
    float* part;            // [tokens * top_k][dim], an expert's output for a token
};

// Elements of a slot's hidden activations (see moe_h_place).
constexpr int64_t moe_h_row(int64_t hidden) {
    return (hidden + kGroup - 1) / kGroup * (2 * kGroup);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Counters have a fixed place, so that calls of different shapes can share a
// workspace.
MoeWs layout(void* ws, int64_t t, int64_t e, int64_t k, int64_t d, int64_t h, size_t* total) {
    uint8_t* p = static_cast<uint8_t*>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t* r = p + at;
        at = up256(at + bytes);
        return r;
    };
    MoeWs w;
    w.route_count = reinterpret_cast<uint32_t*>(take(4 * (kMaxTokens / kRouteTokens)));
    w.group_count = reinterpret_cast<uint32_t*>(take(4));
    w.down_count = reinterpret_cast<uint32_t*>(take(4 * kMaxTokens * (65536 / kRows)));
    w.reached_n = reinterpret_cast<int32_t*>(take(4));
    w.reached = reinterpret_cast<Reached*>(take(sizeof(Reached) * e));
    w.slots = reinterpret_cast<int32_t*>(take(4 * t * k));
    w.logits = reinterpret_cast<float*>(take(4 * t * e));
    w.ids = reinterpret_cast<int32_t*>(take(4 * t * k));
    w.weights = reinterpret_cast<float*>(take(4 * t * k));
    w.h = reinterpret_cast<uint16_t*>(take(2 * t * k * moe_h_row(h)));
    w.part = reinterpret_cast<float*>(take(4 * t * k * d));
    *total = at;
    return w;
}

// Values that workgroups of one launch hand to each other go through memory
// at device scope: stored and loaded there, and a store has reached it when
// the wave's count of outstanding stores is zero.
template <class T>
__device__ __forceinline__ void store_dev(T* p, T v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T load_dev(const T* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void stores_done() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Counts this workgroup in; true in the one that completes `of`, which also
// sets the counter back.  Every lane calls it.
__device__ __forceinline__ bool last_of(uint32_t* counter, uint32_t of, uint32_t* flag) {
    stores_done();
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t seen =
            __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (seen == of - 1)
            __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *flag = seen == of - 1;
    }
    __syncthreads();
    return *flag != 0;
}

// Reductions over a wave by lane permutes inside the vector unit (shifts by
// 1, 2, 4, 8 in rows of 16 lanes, then the rows' last lanes to the next
// rows): the full result is lane 63's.  `id` leaves the other operand as it
// is.
template <class Op>
__device__ __forceinline__ float wave_reduce(float v, float id, Op op) {
    auto step = [&](auto ctrl, auto rows) __attribute__((always_inline)) {
        const int o = __builtin_amdgcn_update_dpp(__float_as_int(id), __float_as_int(v),
                                                  decltype(ctrl)::value, decltype(rows)::value,
                                                  0xf, false);
        v = op(v, __int_as_float(o));
    };
    using std::integral_constant;
    step(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr:1
    step(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
    step(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
    step(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
    step(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});  // row_bcast:15
    step(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});  // row_bcast:31
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float reduce_max(float v) {
    return wave_reduce(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float reduce_sum(float v) {
    return wave_reduce(v, 0.0f, [](float a, float b) { return a + b; });
}

// Top-k of one token by one wave.  Lane l has the logits of experts
// l * PER .. l * PER + PER - 1 (v[], -inf past the last), so the lowest lane
// that holds the maximum, at its first place, is the lowest index.
struct Choice {
    int id;
    float w;
};
template <int PER>
__device__ __forceinline__ Choice select_experts(const MoeLaunch& p, float (&v)[PER], int lane) {
    float mx = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) mx = fmaxf(mx, v[i]);
    mx = reduce_max(mx);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (lane * PER + i < p.experts) sum += expf(v[i] - mx);
    sum = reduce_sum(sum);
    // Bit i: expert i of this lane can still be taken; its logit is NaN.  Those
    // rank below every number, -inf too: they come when no other is left.
    uint32_t left = 0, nan = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (v[i] != v[i]) nan |= 1u << i, v[i] = -INFINITY;
        if (lane * PER + i < p.experts) left |= 1u << i;
    }
    float chosen = -INFINITY;  // lane j's: the j-th expert's logit, and its index
    int chosen_id = 0;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t can = left & ~nan;
        if (__ballot(can != 0) == 0) can = left;
        float best = -INFINITY;
        int at = -1;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if ((can >> i & 1) && (at < 0 || v[i] >= best)) best = v[i], at = i;
        const float top = reduce_max(best);
        const uint64_t who = __ballot(at >= 0 && best == top);
        const int winner = __ffsll((unsigned long long)who) - 1;
        const bool mine = lane == winner;
        float value = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i == at) value = nan >> i & 1 ? NAN : v[i];
        const int id = __builtin_amdgcn_readlane(lane * PER + at, winner);
        value = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(value), winner));
        if (mine) left &= ~(1u << at);
        if (lane == j) chosen = value, chosen_id = id;
    }
    float w = lane < p.top_k ? expf(chosen - mx) / sum : 0.0f;
    if (p.renorm) w /= reduce_sum(w);
    return Choice{chosen_id, w};
}

// Lane j < top_k: the j-th choice of token t.
__device__ __forceinline__ Choice choose(const MoeLaunch& p, const MoeWs& ws, int64_t t,
                                         int lane) {
    auto go = [&](auto per) __attribute__((always_inline)) {
        constexpr int kPer = decltype(per)::value;
        float v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane * kPer + i;
            v[i] = e < p.experts ? load_dev(ws.logits + t * p.experts + e) : -INFINITY;
        }
        return select_experts<kPer>(p, v, lane);
    };
    using std::integral_constant;
    if (p.experts <= kWave) return go(integral_constant<int, 1>{});
    if (p.experts <= 2 * kWave) return go(integral_constant<int, 2>{});
    return go(integral_constant<int, 8>{});
}
__device__ __forceinline__ void store_choice(const MoeLaunch& p, const MoeWs& ws, int64_t t,
                                             int lane, Choice c) {
    if (lane >= p.top_k) return;
    const int64_t o = t * p.top_k + lane;
    store_dev(ws.ids + o, c.id);
    ws.weights[o] = c.w;
    if (p.ids) p.ids[o] = c.id;
    if (p.weights) p.weights[o] = c.w;
}

// The list of reached experts and their slots, by one workgroup.  ids: every
// slot's expert, here already if `have`.
struct Lists {
    uint16_t ids[kMaxTokens * kMaxTopK];
    int count[kMaxExperts], first[kMaxExperts];
    int sums[2][kWaves];
};
__device__ __forceinline__ void build_lists(const MoeLaunch& p, const MoeWs& ws, Lists& s,
                                            bool have) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int n = p.tokens * p.top_k;
    for (int e = tid; e < kMaxExperts; e += kThreads) s.count[e] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        if (!have) s.ids[i] = (uint16_t)load_dev(ws.ids + i);
        atomicAdd(&s.count[s.ids[i]], 1);
    }
    __syncthreads();
    // each thread takes two neighbouring experts: slots and reached ones before them
    static_assert(kMaxExperts == 2 * kThreads, "two experts per thread");
    const int c0 = s.count[2 * tid], c1 = s.count[2 * tid + 1];
    int slots = c0 + c1, used = (c0 > 0) + (c1 > 0);
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int a = __shfl_up(slots, off, kWave), b = __shfl_up(used, off, kWave);
        if (lane >= off) slots += a, used += b;
    }
    if (lane == kWave - 1) s.sums[0][wave] = slots, s.sums[1][wave] = used;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) slots += s.sums[0][w], used += s.sums[1][w];
        all += s.sums[1][w];
    }
    const int f0 = slots - c0 - c1, f1 = slots - c1;
    int u = used - (c0 > 0) - (c1 > 0);
    if (c0 > 0) ws.reached[u++] = Reached{2 * tid, f0, c0, 0};
    if (c1 > 0) ws.reached[u] = Reached{2 * tid + 1, f1, c1, 0};
    s.first[2 * tid] = f0;
    s.first[2 * tid + 1] = f1;
    if (tid == 0) *ws.reached_n = all;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
        ws.slots[atomicAdd(&s.first[s.ids[i]], 1)] = i;
}

// A workgroup computes the logits of 4 experts (one a wave) for 4 tokens;
// the last of a token group's workgroups selects its experts (a token a
// wave), and the last of those writes the lists.
__global__ __launch_bounds__(kThreads) void moe_route_kernel(MoeLaunch p, MoeWs ws) {
    static_assert(kRouteTokens == kWaves, "a token per wave");
    __shared__ Lists lists;
    __shared__ uint32_t flag;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int t0 = blockIdx.y * kRouteTokens;
    const int e = blockIdx.x * kWaves + wave;
    if (e < p.experts) {
        const uint16_t* r = p.router + (int64_t)e * p.dim;
        const uint16_t* x[kRouteTokens];
        float acc[kRouteTokens];
#pragma unroll
        for (int i = 0; i < kRouteTokens; ++i) {
            // (past the last token: the last again, not stored)
            const int t = t0 + i < p.tokens ? t0 + i : p.tokens - 1;
            x[i] = p.x + (int64_t)t * p.dim;
            acc[i] = 0.0f;
        }
        // 2048 k a round, all their loads ahead of the first product; lanes past
        // dim (a multiple of 16) read what exists and drop it
        constexpr int kStep = 8 * kWave, kAhead = 4;
        for (int d0 = 0; d0 < p.dim; d0 += kAhead * kStep) {
            uint4 rv[kAhead], xv[kAhead][kRouteTokens];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int d = d0 + a * kStep + 8 * lane;
                const int at = d < p.dim ? d : 0;
                rv[a] = *reinterpret_cast<const uint4*>(r + at);
#pragma unroll
                for (int i = 0; i < kRouteTokens; ++i)
                    xv[a][i] = *reinterpret_cast<const uint4*>(x[i] + at);
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (d0 + a * kStep + 8 * lane >= p.dim) continue;
                const uint32_t rw[4] = {rv[a].x, rv[a].y, rv[a].z, rv[a].w};
#pragma unroll
                for (int i = 0; i < kRouteTokens; ++i) {
                    const uint32_t xw[4] = {xv[a][i].x, xv[a][i].y, xv[a][i].z, xv[a][i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[i] = fmaf(bf16_lo(xw[j]), bf16_lo(rw[j]), acc[i]);
                        acc[i] = fmaf(bf16_hi(xw[j]), bf16_hi(rw[j]), acc[i]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRouteTokens; ++i) {
            const float s = reduce_sum(acc[i]);
            if (lane == 0 && t0 + i < p.tokens)
                store_dev(ws.logits + (int64_t)(t0 + i) * p.experts + e, s);
        }
    }
    if (p.tokens == 1) return;  // the next launch's workgroups choose
    if (!last_of(ws.route_count + blockIdx.y, gridDim.x, &flag)) return;
    const int t = t0 + wave;
    if (t < p.tokens) {
        const Choice c = choose(p, ws, t, lane);
        if (lane < p.top_k) lists.ids[wave * p.top_k + lane] = (uint16_t)c.id;
        store_choice(p, ws, t, lane, c);
    }
    const bool all = gridDim.y == 1;  // this workgroup chose for every token
    if (all) __syncthreads();
    else if (!last_of(ws.group_count, gridDim.y, &flag)) return;
    build_lists(p, ws, lists, all);
}

// Eight fp8 codes -> bf16 (exact).
template <int FMT>
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
    bf16x8 r;
    auto put = [&](int at, uint32_t w) __attribute__((always_inline)) {
        bf16x2_t a, b;
        if constexpr (FMT) {
            a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, false);
            b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, true);
        } else {
            a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
            b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
        }
        r[at] = a[0];
        r[at + 1] = a[1];
        r[at + 2] = b[0];
        r[at + 3] = b[1];
    };
    put(0, lo);
    put(4, hi);
    return r;
}

__device__ __forceinline__ v4f mfma_bf16(const bf16x8& a, const bf16x8& b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8 as_bf16(const uint4& v) {
    return __builtin_bit_cast(bf16x8, v);
}

typedef uint32_t vec4 __attribute__((ext_vector_type(4)));

// Four fp8 codes -> fp32 (exact).
template <int FMT>
__device__ __forceinline__ void fp8_to_f32(uint32_t w, float (&f)[4]) {
    if constexpr (FMT) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
        f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1];
    } else {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1];
    }
}

// kTiles 16-row tiles of weights times the activations of 16 tokens over the
// 128-k blocks wave, wave + 4, ... of `kdim`: acc[tile] += step * sum.
//
// A load takes whole 128-byte lines of 8 rows (lane l: row l % 8, bytes 16 (l / 8)
// ..); with loads of 16 rows x 64 bytes, as the matrix instruction has them, 64
// tokens took 124 us instead of 109.  With STREAM the loads go past the caches: a gain
// where an expert has up to 16 tokens and so each weight is read once (64 tokens,
// 8 of 64 experts of 2048 x 1024, 100 us, 105 without), a loss where it is read
// again (64 tokens that all take 8 of 8 experts 84 us, 80 without; 256 tokens, 8 of
// 64, 272 and 245).  Not where kdim is no multiple of 128, since a row's pieces then
// share lines (13 tokens, 1040 x 688: 25.3 us, 29.0 with).
// Between a tile's two loads lanes l and l ^ 8 then exchange halves, by one lane permute
// per register, so that lane l holds row l % 16 and k = 32 (l / 16) .. + 31 of
// the block: a reordering of k that the sum does not see.
//   w[tile]: the tile's first row;  s[tile]: its steps (both uniform).
//   act, at: this lane's token's activations begin at element `at`; H: they
//   are hidden activations, as moe_h_place lays them out.  AHEAD: one block's
//   loads go out before the block before it is multiplied (see kManyGroups).
template <int FMT, bool H, bool STREAM, bool AHEAD>
__device__ __forceinline__ void tile_products(const uint8_t* const (&w)[kTiles],
                                              const float* const (&s)[kTiles],
                                              const uint16_t* act, uint32_t at, int kdim,
                                              int wave, int lane, v4f (&acc)[kTiles]) {
    constexpr int kParts = H ? 2 : 1;  // a hidden activation's two numbers
    const int wk = 16 * (lane / 8), xk = 32 * (lane / 16);
    const uint32_t wo = (uint32_t)((lane % 8) * kdim + wk);
    const uint32_t xo = 2 * (at + (H ? 8 * (lane / 16) : xk));
    struct Block {
        vec4 w[kTiles][2];
        uint4 x[kParts][4];
        float s[kTiles];
    };
    auto load = [&](int n, Block& b) __attribute__((always_inline)) {
        const int k0 = kGroup * n;
        const bool whole = k0 + kGroup <= kdim;  // uniform
        // kdim is a multiple of 16: a lane's 16 k of a load exist or none does
        // (one that exists instead)
        const uint32_t wat = wo + (whole || k0 + wk < kdim ? k0 : -wk);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const vec4* src = reinterpret_cast<const vec4*>(w[t] + 8 * i * kdim + wat);
                if constexpr (STREAM) b.w[t][i] = __builtin_nontemporal_load(src);
                else b.w[t][i] = *src;
            }
#pragma unroll
        for (int a = 0; a < kParts; ++a)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t x;
                if constexpr (H) x = xo + 4 * k0 + 256 * a + 64 * j;
                else x = xo + (whole || k0 + xk + 8 * j < kdim ? 2 * k0 + 16 * j : -2 * xk);
                b.x[a][j] = *reinterpret_cast<const uint4*>(
                    reinterpret_cast<const uint8_t*>(act) + x);
            }
        if (!whole) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (k0 + wk >= kdim) b.w[t][i] = vec4{0, 0, 0, 0};
#pragma unroll
            for (int a = 0; a < kParts; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k0 + xk + 8 * j >= kdim) b.x[a][j] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) b.s[t] = s[t][n];
    };
    auto multiply = [&](const Block& b) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            vec4 f[2];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int w0 = (int)b.w[t][0][d], w1 = (int)b.w[t][1][d];
                // row_ror:8 into lanes 8 .. 15, and into 0 .. 7, of each 16
                f[0][d] = (uint32_t)__builtin_amdgcn_update_dpp(w0, w1, 0x128, 0xf, 0xc, false);
                f[1][d] = (uint32_t)__builtin_amdgcn_update_dpp(w1, w0, 0x128, 0xf, 0x3, false);
            }
            v4f part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 m = widen<FMT>(f[j / 2][2 * (j % 2)], f[j / 2][2 * (j % 2) + 1]);
#pragma unroll
                for (int a = 0; a < kParts; ++a) part = mfma_bf16(m, as_bf16(b.x[a][j]), part);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(part[i], b.s[t], acc[t][i]);
        }
    };
    const int blocks = (kdim + kGroup - 1) / kGroup;
    if constexpr (!AHEAD) {
        for (int b = wave; b < blocks; b += kWaves) {
            Block k;
            load(b, k);
            multiply(k);
        }
        return;
    }
    if (wave >= blocks) return;
    Block one, two;
    load(wave, one);
    for (int b = wave; b < blocks; b += 2 * kWaves) {
        if (b + kWaves < blocks) load(b + kWaves, two);
        multiply(one);
        if (b + 2 * kWaves < blocks) load(b + 2 * kWaves, one);
        if (b + kWaves < blocks) multiply(two);
    }
}

// Hidden activations lie as the down kernel's loads take them: a row of
// moe_h_row elements per slot, of each 128 units the rounded numbers and then
// the rests, unit 32 q + 8 j + e of them at 32 j + 8 q + e.
__device__ __forceinline__ int moe_h_place(int f) {
    const int r = f % kGroup;
    return f / kGroup * (2 * kGroup) + 32 * (r / 8 % 4) + 8 * (r / 32) + r % 8;
}

// The waves' sums of a kTiles x 16 x 16 result, added in wave order: thread
// (token = tid / 16, row = tid % 16) gets every tile's value.  acc[t][i] is
// row 4 (lane / 16) + i, token lane % 16.
typedef float Partial[kWaves][kTiles][16][17];
__device__ __forceinline__ void join_waves(const v4f (&acc)[kTiles], Partial& red,
                                           float (&out)[kTiles]) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][t][lane % 16][4 * (lane / 16) + i] = acc[t][i];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        float v = red[0][t][tid / 16][tid % 16];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][t][tid / 16][tid % 16];
        out[t] = v;
    }
    __syncthreads();
}

// ONE: there is one token, whose top_k choices each workgroup makes for itself
// from the logits that the launch before left, and takes the blockIdx.y-th.
// That is cheaper than choosing before, in the last workgroup to bring its
// logits: two round trips through memory and the lists.
template <int FMT, bool STREAM, bool AHEAD, bool ONE>
__global__ __launch_bounds__(kThreads) void moe_gate_up_kernel(MoeLaunch p, MoeWs ws) {
    __shared__ Partial red;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    Reached work;
    if constexpr (ONE) {
        const Choice c = choose(p, ws, 0, lane);
        work = Reached{__builtin_amdgcn_readlane(c.id, blockIdx.y), (int)blockIdx.y, 1, 0};
        if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) store_choice(p, ws, 0, lane, c);
    } else {
        if ((int)blockIdx.y >= *ws.reached_n) return;
        work = ws.reached[blockIdx.y];
    }
    const int64_t e = work.expert;
    const int f0 = blockIdx.x * kUnits;
    const int kg = (p.dim + kGroup - 1) / kGroup, rg = (2 * p.hidden + kGroup - 1) / kGroup;
    constexpr int kHalf = kTiles / 2;  // tiles of gate rows, then as many of up rows
    const uint8_t* w[kTiles];
    const float* s[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        // 16 rows share a tile of steps (hidden is a multiple of 16); a second
        // 16 units past the last repeat the first
        const int f = f0 + 16 * (t % kHalf) < p.hidden ? f0 + 16 * (t % kHalf) : f0;
        const int row = f + t / kHalf * p.hidden;
        w[t] = p.w13 + (e * 2 * p.hidden + row) * p.dim;
        s[t] = p.s13 + (e * rg + row / kGroup) * kg;
    }
    for (int c0 = 0; c0 < work.count; c0 += 16) {
        // lanes past the list repeat its last token; their results are dropped
        const int c = c0 + lane % 16 < work.count ? c0 + lane % 16 : work.count - 1;
        const int slot = ONE ? work.first : ws.slots[work.first + c];
        v4f acc[kTiles] = {};
        tile_products<FMT, false, STREAM, AHEAD>(
            w, s, p.x, (uint32_t)(slot / p.top_k * p.dim), p.dim, wave, lane, acc);
        float v[kTiles];
        join_waves(acc, red, v);
        if (c0 + tid / 16 < work.count) {
            const int at_slot = ONE ? work.first : ws.slots[work.first + c0 + tid / 16];
            uint16_t* row = ws.h + at_slot * moe_h_row(p.hidden);
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                const float h = v[i] / (1.0f + expf(-v[i])) * v[kHalf + i];
                // Finite values that round past bf16's largest keep that and the
                // rest; an infinite one has no rest (inf - inf is NaN).
                const bool inf = fabsf(h) == INFINITY;
                uint16_t hi = f32_to_bf16(h);
                if ((hi & 0x7fff) == 0x7f80 && !inf) --hi;
                if (f0 + 16 * i < p.hidden) {
                    uint16_t* at = row + moe_h_place(f0 + 16 * i + tid % 16);
                    at[0] = hi;
                    at[kGroup] = inf ? 0 : f32_to_bf16(h - bf16_to_f32(hi));
                }
            }
        }
    }
}

// A workgroup's outputs for a token are one expert's share; the workgroup
// that brings the last of the token's shares for these rows adds them up, in
// the order of the token's choices (so the result does not depend on which
// came last).
template <int FMT, bool STREAM, bool AHEAD>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeLaunch p, MoeWs ws) {
    __shared__ Partial red;
    __shared__ int done[16];  // tokens of this round that are complete, else -1
    if ((int)blockIdx.y >= *ws.reached_n) return;
    const Reached work = ws.reached[blockIdx.y];
    const int64_t e = work.expert;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int d0 = blockIdx.x * kRows;
    const int kg = (p.hidden + kGroup - 1) / kGroup, rg = (p.dim + kGroup - 1) / kGroup;
    const uint8_t* w[kTiles];
    const float* s[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        // dim is a multiple of 16: a tile past it repeats the first
        const int row = d0 + 16 * t < p.dim ? d0 + 16 * t : d0;
        w[t] = p.w2 + (e * p.dim + row) * p.hidden;
        s[t] = p.s2 + (e * rg + row / kGroup) * kg;
    }
    for (int c0 = 0; c0 < work.count; c0 += 16) {
        const int c = c0 + lane % 16 < work.count ? c0 + lane % 16 : work.count - 1;
        const uint32_t at = (uint32_t)(ws.slots[work.first + c] * moe_h_row(p.hidden));
        v4f acc[kTiles] = {};
        tile_products<FMT, true, STREAM, AHEAD>(w, s, ws.h, at, p.hidden, wave, lane, acc);
        float v[kTiles];
        join_waves(acc, red, v);
        if (c0 + tid / 16 < work.count) {
            float* o = ws.part + (int64_t)ws.slots[work.first + c0 + tid / 16] * p.dim + d0 +
                       tid % 16;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                if (d0 + 16 * t < p.dim) store_dev(o + 16 * t, v[t]);
        }
        stores_done();
        __syncthreads();
        if (tid < 16) {
            int complete = -1;
            if (c0 + tid < work.count) {
                const int t = ws.slots[work.first + c0 + tid] / p.top_k;
                uint32_t* n = ws.down_count + (int64_t)blockIdx.x * kMaxTokens + t;
                const uint32_t seen = __hip_atomic_fetch_add(n, 1u, __ATOMIC_RELAXED,
                                                             __HIP_MEMORY_SCOPE_AGENT);
                if (seen == (uint32_t)p.top_k - 1) {
                    complete = t;
                    store_dev(n, 0u);
                }
            }
            done[tid] = complete;
        }
        __syncthreads();
        // two outputs a thread, 8 tokens at a time, eight loads in flight
        const int d = d0 + 2 * (tid % (kRows / 2));
        for (int i = tid / (kRows / 2); i < 16; i += kThreads / (kRows / 2)) {
            const int t = done[i];
            if (t < 0 || d >= p.dim) continue;
            float y0 = 0.0f, y1 = 0.0f;
            for (int j0 = 0; j0 < p.top_k; j0 += 8) {
                uint64_t u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int64_t slot = (int64_t)t * p.top_k + (j0 + j < p.top_k ? j0 + j : j0);
                    u[j] = load_dev(reinterpret_cast<const uint64_t*>(ws.part + slot * p.dim + d));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (j0 + j >= p.top_k) break;
                    const float g = ws.weights[(int64_t)t * p.top_k + j0 + j];
                    y0 = fmaf(g, __uint_as_float((uint32_t)u[j]), y0);
                    y1 = fmaf(g, __uint_as_float((uint32_t)(u[j] >> 32)), y1);
                }
            }
            *reinterpret_cast<uint32_t*>(p.out + (int64_t)t * p.dim + d) = f32x2_to_bf16x2(y0, y1);
        }
    }
}

// One token: a workgroup owns kOneRows outputs, a wave of it one choice (or,
// where there are few, a share of its blocks) at a time, so the shares meet in
// LDS and not in memory.  Lane l has 16 k from 16 (l % 8) on of row l / 8 of each
// block of 128, whose sum times the step is added in fp32; the matrix unit has nothing to share between tokens here.
template <int FMT>
__global__ __launch_bounds__(kOneWaves * kWave) void moe_down_one_kernel(MoeLaunch p, MoeWs ws) {
    static_assert(kOneRows == kWave / 8, "8 lanes a row");
    __shared__ float red[kMaxTopK][kOneRows];
    const int tid = threadIdx.x, lane = tid % kWave, c = lane % 8, r = lane / 8;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int d0 = blockIdx.x * kOneRows;
    const int kg = (p.hidden + kGroup - 1) / kGroup, rg = (p.dim + kGroup - 1) / kGroup;
    // a choice's blocks go to several waves when there are few choices
    const int parts = p.top_k < kOneWaves ? kOneWaves / p.top_k : 1;
    for (int task = wave; task < p.top_k * parts; task += kOneWaves) {
        const int j = task / parts, part_of = task % parts;
        const int first = kg * part_of / parts, last = kg * (part_of + 1) / parts;
        const int64_t e = ws.ids[j];
        const uint8_t* w = p.w2 + (e * p.dim + d0) * p.hidden + (r * p.hidden + 16 * c);
        const float* s = p.s2 + (e * rg + d0 / kGroup) * kg;
        // (moe_h_place of the lane's first unit in a block)
        const uint16_t* h = ws.h + j * moe_h_row(p.hidden) + 64 * (c % 2) + 8 * (c / 2);
        float acc = 0.0f;
        constexpr int kBlocks = 2;  // in flight (one or three: 1.5 us more)
        for (int b0 = first; b0 < last; b0 += kBlocks) {
            vec4 wv[kBlocks];
            uint4 hv[kBlocks][4];
            float step[kBlocks];
            bool ok[kBlocks];
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                // all of the lane's 16 k exist, or none (something that exists instead)
                ok[i] = b0 + i < last && kGroup * (b0 + i) + 16 * c < p.hidden;
                const int b = b0 + i < last ? b0 + i : 0;
                wv[i] = __builtin_nontemporal_load(
                    reinterpret_cast<const vec4*>(w + (ok[i] ? kGroup * (b0 + i) : -16 * c)));
#pragma unroll
                for (int q = 0; q < 4; ++q)  // numbers, and from 128 on their rests
                    hv[i][q] = *reinterpret_cast<const uint4*>(h + 2 * kGroup * b +
                                                               kGroup * (q / 2) + 32 * (q % 2));
                step[i] = s[b];
            }
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                float part = 0.0f;
#pragma unroll
                for (int q = 0; q < 2; ++q) {  // 8 k
                    const uint32_t hi[4] = {hv[i][q].x, hv[i][q].y, hv[i][q].z, hv[i][q].w};
                    const uint32_t lo[4] = {hv[i][2 + q].x, hv[i][2 + q].y, hv[i][2 + q].z,
                                            hv[i][2 + q].w};
                    float hf[8];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        hf[2 * x] = bf16_lo(hi[x]) + bf16_lo(lo[x]);
                        hf[2 * x + 1] = bf16_hi(hi[x]) + bf16_hi(lo[x]);
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float f[4];
                        fp8_to_f32<FMT>(wv[i][2 * q + x], f);
#pragma unroll
                        for (int z = 0; z < 4; ++z) part = fmaf(f[z], hf[4 * x + z], part);
                    }
                }
                // (kept out of a branch, into which its loads would go too)
                float sum = fmaf(part, step[i], acc);
                asm volatile("" : "+v"(sum));
                acc = ok[i] ? sum : acc;
            }
        }
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) acc += __shfl_xor(acc, off, kWave);
        if (c == 0) red[task][r] = acc;
    }
    __syncthreads();
    if (tid < kOneRows / 2) {
        float y0 = 0.0f, y1 = 0.0f;
        for (int j = 0; j < p.top_k; ++j) {
            const float g = ws.weights[j];
            float s0 = 0.0f, s1 = 0.0f;
            for (int i = j * parts; i < (j + 1) * parts; ++i) {
                s0 += red[i][2 * tid];
                s1 += red[i][2 * tid + 1];
            }
            y0 = fmaf(g, s0, y0);
            y1 = fmaf(g, s1, y1);
        }
        *reinterpret_cast<uint32_t*>(p.out + d0 + 2 * tid) = f32x2_to_bf16x2(y0, y1);
    }
}

}  // namespace

size_t moe_workspace(int64_t tokens, int64_t experts, int64_t top_k, int64_t dim, int64_t hidden) {
    size_t total;
    layout(nullptr, tokens, experts, top_k, dim, hidden, &total);
    return total;
}

hipError_t launch_moe(const MoeLaunch& p, hipStream_t stream) {
    size_t total;
    const MoeWs ws = layout(p.ws, p.tokens, p.experts, p.top_k, p.dim, p.hidden, &total);
    hipLaunchKernelGGL(moe_route_kernel,
                       dim3((p.experts + kWaves - 1) / kWaves,
                            (p.tokens + kRouteTokens - 1) / kRouteTokens),
                       dim3(kThreads), 0, stream, p, ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int slots = p.tokens * p.top_k;
    const int reach = slots < p.experts ? slots : p.experts;  // at most so many experts
    const dim3 up((p.hidden + kUnits - 1) / kUnits, reach);
    const dim3 down((p.dim + kRows - 1) / kRows, reach);
    using std::bool_constant;
    auto gate_up = [&](auto fmt, auto stream_c, auto ahead) {
        hipLaunchKernelGGL((moe_gate_up_kernel<decltype(fmt)::value, decltype(stream_c)::value,
                                               decltype(ahead)::value, false>),
                           up, dim3(kThreads), 0, stream, p, ws);
        return hipGetLastError();
    };
    auto down_all = [&](auto fmt, auto stream_c, auto ahead) {
        hipLaunchKernelGGL((moe_down_kernel<decltype(fmt)::value, decltype(stream_c)::value,
                                            decltype(ahead)::value>),
                           down, dim3(kThreads), 0, stream, p, ws);
        return hipGetLastError();
    };
    auto pick = [&](auto launch_one, auto fmt, int kdim, dim3 grid) {
        const bool ahead = grid.x * grid.y < kManyGroups;
        if (kdim % kGroup == 0)
            return ahead ? launch_one(fmt, bool_constant<true>{}, bool_constant<true>{})
                         : launch_one(fmt, bool_constant<true>{}, bool_constant<false>{});
        return ahead ? launch_one(fmt, bool_constant<false>{}, bool_constant<true>{})
                     : launch_one(fmt, bool_constant<false>{}, bool_constant<false>{});
    };
    // One token, us, against the form for more: 64 experts of 2048 x 1024, 8 a
    // token, 22.7 / 25.3; 32 of 1040 x 688, 2, 14.4 / 19.2; 16 of 4096 x 2048, 4,
    // 36.0 / 36.1; 8 of 4096 x 4096, 2, 35.2 / 40.8.  The same form for two tokens,
    // which read shared experts twice then, 31.0 / 33.3 and 16.3 / 19.6, but 57.1 /
    // 51.7 and 63.6 / 52.2.
    auto launch_one = [&](auto fmt) {
        constexpr int kFmt = decltype(fmt)::value;
        auto* up_kernel = p.dim % kGroup == 0 ? moe_gate_up_kernel<kFmt, true, true, true>
                                              : moe_gate_up_kernel<kFmt, false, true, true>;
        hipLaunchKernelGGL(up_kernel, up, dim3(kThreads), 0, stream, p, ws);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        hipLaunchKernelGGL((moe_down_one_kernel<kFmt>), dim3(p.dim / kOneRows),
                           dim3(kOneWaves * kWave), 0, stream, p, ws);
        return hipGetLastError();
    };
    auto launch = [&](auto fmt) {
        if (p.tokens == 1) return launch_one(fmt);
        const hipError_t err = pick(gate_up, fmt, p.dim, up);
        return err == hipSuccess ? pick(down_all, fmt, p.hidden, down) : err;
    };
    return p.fmt == 0 ? launch(std::integral_constant<int, 0>{})
                      : launch(std::integral_constant<int, 1>{});
}

}  // namespace fp8lin
