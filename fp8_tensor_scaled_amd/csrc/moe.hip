// Mixture-of-experts layer for a few tokens on tile-scaled fp8 weights:
//   l = x R^T;  the top_k experts e_j of each token (ties: lowest index);
//   w = softmax(l)[e_j], over their sum when asked;
//   y = sum_j w_j W2_e ( silu(G_e x) * (U_e x) ),  every weight = code * step.
//
// With few tokens per expert the layer is bound by reading the chosen
// experts' weights once (3 dim hidden bytes each), so both products are
// shaped for that:
//
//  * A workgroup takes 16 hidden units of one expert (16 rows of G and of U)
//    or 32 rows of W2, for all of the expert's tokens; its 4 waves take the
//    128-k blocks in turn, so every byte of x and of the weights is loaded by
//    one wave of it, and the four partial sums meet in LDS in a fixed order.
//  * Weights go straight into registers in the matrix instruction's layout
//    (16 rows x 64 bytes per load), one block ahead, are widened to bf16
//    (exact) and multiplied by bf16 activations: 16 tokens ride on one
//    16x16x32 instruction, so one token costs what 16 do.
//  * A block of 128 k lies in one tile of steps: its four instructions start
//    from zero, and the sum times the step is added in fp32.
//  * The hidden activations go between the two kernels as two bf16 numbers
//    each (the value rounded, and the rest rounded): 16 bits of precision
//    for one more matrix instruction, which the loads hide.

#include "block.hpp"
#include "common.hpp"

namespace fp8lin {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxExperts = 512, kMaxTokens = 1024;
constexpr int kRouteTokens = 8;   // tokens of a routing workgroup
constexpr int kUnits = 16;        // hidden units of a gate / up workgroup
constexpr int kRows = 32;         // rows of W2 of a down workgroup

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Workspace: counters first (zero between calls), then what one kernel
// leaves for the next.
struct MoeWs {
    uint32_t* route_count;  // per token group: routing workgroups done
    uint32_t* down_count;   // per 32 rows of the output: experts done
    float* logits;          // [tokens][experts]
    int32_t* ids;           // [tokens][top_k]
    float* weights;         // [tokens][top_k]
    uint16_t* h_hi;         // bf16 [tokens * top_k][hidden]
    uint16_t* h_lo;
    float* part;            // [tokens * top_k][dim], an expert's output for a token
};

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Counters have a fixed place, so that calls of different shapes can share a
// workspace: kMaxTokens / kRouteTokens and 65536 / kRows words.
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
    w.down_count = reinterpret_cast<uint32_t*>(take(4 * (65536 / kRows)));
    w.logits = reinterpret_cast<float*>(take(4 * t * e));
    w.ids = reinterpret_cast<int32_t*>(take(4 * t * k));
    w.weights = reinterpret_cast<float*>(take(4 * t * k));
    w.h_hi = reinterpret_cast<uint16_t*>(take(2 * t * k * h));
    w.h_lo = reinterpret_cast<uint16_t*>(take(2 * t * k * h));
    w.part = reinterpret_cast<float*>(take(4 * t * k * d));
    *total = at;
    return w;
}

// Values that workgroups of one launch hand to each other go through memory
// at device scope: stored and loaded there, and a store has reached it when
// the wave's count of outstanding stores is zero.
__device__ __forceinline__ void store_dev(float* p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_dev(const float* p) {
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

// Top-k of one token by one wave: logits in LDS.
__device__ __forceinline__ void select_experts(const MoeLaunch& p, const MoeWs& ws, int64_t t,
                                               const float* logit, int lane) {
    float mx = -INFINITY, sum = 0.0f;
    for (int e = lane; e < p.experts; e += kWave) mx = fmaxf(mx, logit[e]);
    mx = wave_max(mx);
    for (int e = lane; e < p.experts; e += kWave) sum += expf(logit[e] - mx);
    sum = wave_sum(sum);
    uint32_t taken = 0;  // bit i: this lane's expert lane + 64 i is taken
    float chosen = 0.0f, total = 0.0f;
    int chosen_id = 0;
    for (int j = 0; j < p.top_k; ++j) {
        float best = -INFINITY;
        int at = kMaxExperts;  // NaN and -inf logits lose to any other, lowest index first
        for (int e = lane, i = 0; e < p.experts; e += kWave, ++i) {
            if (taken >> i & 1) continue;
            const float v = logit[e] == logit[e] ? logit[e] : -INFINITY;
            if (at == kMaxExperts || v > best) best = v, at = e;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const float ov = __shfl_xor(best, off, kWave);
            const int oa = __shfl_xor(at, off, kWave);
            if (oa < kMaxExperts && (at == kMaxExperts || ov > best || (ov == best && oa < at)))
                best = ov, at = oa;
        }
        if (at % kWave == lane) taken |= 1u << (at / kWave);
        const float w = expf(logit[at] - mx) / sum;
        total += w;
        if (lane == j) chosen = w, chosen_id = at;
    }
    if (lane < p.top_k) {
        const float w = p.renorm ? chosen / total : chosen;
        const int64_t o = t * p.top_k + lane;
        ws.ids[o] = chosen_id;
        ws.weights[o] = w;
        if (p.ids) p.ids[o] = chosen_id;
        if (p.weights) p.weights[o] = w;
    }
}

// A workgroup computes the logits of 4 experts (one a wave) for 8 tokens;
// the last of a token group's workgroups selects its experts.
__global__ __launch_bounds__(kThreads) void moe_route_kernel(MoeLaunch p, MoeWs ws) {
    __shared__ float logit[kWaves][kMaxExperts];
    __shared__ uint32_t flag;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int t0 = blockIdx.y * kRouteTokens;
    const int nt = p.tokens - t0 < kRouteTokens ? p.tokens - t0 : kRouteTokens;
    const int e = blockIdx.x * kWaves + wave;
    if (e < p.experts) {
        float acc[kRouteTokens];
#pragma unroll
        for (int i = 0; i < kRouteTokens; ++i) acc[i] = 0.0f;
        const uint16_t* r = p.router + (int64_t)e * p.dim;
        const uint16_t* x = p.x + (int64_t)t0 * p.dim;
        for (int d = 8 * lane; d < p.dim; d += 8 * kWave) {  // dim is a multiple of 16
            const uint4 rv = *reinterpret_cast<const uint4*>(r + d);
            const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
            for (int i = 0; i < kRouteTokens; ++i) {
                if (i >= nt) break;
                const uint4 xv = *reinterpret_cast<const uint4*>(x + (int64_t)i * p.dim + d);
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i] = fmaf(bf16_lo(xw[j]), bf16_lo(rw[j]), acc[i]);
                    acc[i] = fmaf(bf16_hi(xw[j]), bf16_hi(rw[j]), acc[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRouteTokens; ++i) {
            if (i >= nt) break;
            const float s = wave_sum(acc[i]);
            if (lane == 0) store_dev(ws.logits + (int64_t)(t0 + i) * p.experts + e, s);
        }
    }
    if (!last_of(ws.route_count + blockIdx.y, gridDim.x, &flag)) return;
    for (int i = wave; i < nt; i += kWaves) {
        for (int j = lane; j < p.experts; j += kWave)
            logit[wave][j] = load_dev(ws.logits + (int64_t)(t0 + i) * p.experts + j);
        // one wave writes and reads these: its LDS accesses are in order
        select_experts(p, ws, t0 + i, logit[wave], lane);
    }
}

// The u-th expert (by index) that any token chose, and its slots (token *
// top_k + rank) in order.  Every lane calls it; -1: there are fewer.
struct Picked {
    uint32_t mask[kMaxExperts / 32];
    uint32_t wave_count[kWaves];
    uint16_t slot[kMaxTokens];
};
__device__ __forceinline__ int pick_expert(const int32_t* ids, int n, int u, Picked& s,
                                           int& count, int& reached) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    if (tid < kMaxExperts / 32) s.mask[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const int e = ids[i];
        atomicOr(&s.mask[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    int expert = -1, before = 0;
    for (int w = 0; w < kMaxExperts / 32; ++w) {
        uint32_t m = s.mask[w];
        const int c = __popc(m);
        if (u >= before && u < before + c) {
            for (int skip = u - before; skip > 0; --skip) m &= m - 1;
            expert = 32 * w + __ffs(m) - 1;
        }
        before += c;
    }
    reached = before;
    if (expert < 0) return -1;
    // each wave takes a quarter of the slots, in order
    const int per = (n + kThreads - 1) / kThreads * kWave;
    const int b = wave * per, e = b + per < n ? b + per : n;
    int c = 0;
    for (int i = b; i < e; i += kWave)
        c += __popcll(__ballot(i + lane < e && ids[i + lane] == expert));
    if (lane == 0) s.wave_count[wave] = c;
    __syncthreads();
    int at = 0;
    count = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) at += s.wave_count[w];
        count += s.wave_count[w];
    }
    for (int i = b; i < e; i += kWave) {
        const bool hit = i + lane < e && ids[i + lane] == expert;
        const uint64_t m = __ballot(hit);
        if (hit) s.slot[at + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(i + lane);
        at += __popcll(m);
    }
    __syncthreads();
    return expert;
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

// Two 16-row tiles of weights times the activations of 16 tokens over the
// 128-k blocks wave, wave + 4, ... of `kdim`: acc[tile] += step * sum.
// Lane l holds rows l % 16 and k = 64 i + 16 (l / 16) .. + 15 of a block (i =
// 0, 1) on both sides, which is a reordering of k that the sum does not see.
//   w[tile]: this lane's row at its first k;  s[tile]: the tile's steps.
//   act[ACT]: the token's activations (added: the lane's rest, if any).
template <int FMT, int ACT>
__device__ __forceinline__ void tile_products(const uint8_t* const (&w)[2],
                                              const float* const (&s)[2],
                                              const uint16_t* const (&act)[ACT], int kdim,
                                              int wave, int lane, v4f (&acc)[2]) {
    const int kq = 16 * (lane / 16);
    struct Block {
        uint4 w[2][2];
        uint4 x[ACT][2][2];
        float s[2];
    };
    auto load = [&](int b, Block& k) __attribute__((always_inline)) {
        const bool whole = kGroup * (b + 1) <= kdim;  // uniform
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k0 = kGroup * b + 64 * i;
            // kdim is a multiple of 16: a lane's 16 k exist or none does
            const bool in = whole || k0 + kq < kdim;
            const int at = in ? k0 : -kq;  // (one that exists instead)
#pragma unroll
            for (int t = 0; t < 2; ++t) k.w[t][i] = *reinterpret_cast<const uint4*>(w[t] + at);
#pragma unroll
            for (int a = 0; a < ACT; ++a) {
                k.x[a][i][0] = *reinterpret_cast<const uint4*>(act[a] + at);
                k.x[a][i][1] = *reinterpret_cast<const uint4*>(act[a] + at + 8);
            }
            if (!whole) {
                auto keep = [&](uint4& v) __attribute__((always_inline)) {
                    v.x = in ? v.x : 0u;
                    v.y = in ? v.y : 0u;
                    v.z = in ? v.z : 0u;
                    v.w = in ? v.w : 0u;
                };
#pragma unroll
                for (int t = 0; t < 2; ++t) keep(k.w[t][i]);
#pragma unroll
                for (int a = 0; a < ACT; ++a) keep(k.x[a][i][0]), keep(k.x[a][i][1]);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) k.s[t] = s[t][b];
    };
    auto multiply = [&](const Block& k) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            v4f part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bf16x8 lo = widen<FMT>(k.w[t][i].x, k.w[t][i].y);
                const bf16x8 hi = widen<FMT>(k.w[t][i].z, k.w[t][i].w);
#pragma unroll
                for (int a = 0; a < ACT; ++a) {
                    part = mfma_bf16(lo, as_bf16(k.x[a][i][0]), part);
                    part = mfma_bf16(hi, as_bf16(k.x[a][i][1]), part);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(part[i], k.s[t], acc[t][i]);
        }
    };
    const int blocks = (kdim + kGroup - 1) / kGroup;
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

// The waves' sums of a 2 x 16 x 16 result, added in wave order: thread
// (token = tid / 16, row = tid % 16) gets both tiles' values.  acc[t][i] is
// row 4 (lane / 16) + i, token lane % 16.
typedef float Partial[kWaves][2][16][17];
__device__ __forceinline__ void join_waves(const v4f (&acc)[2], Partial& red, float (&out)[2]) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][t][lane % 16][4 * (lane / 16) + i] = acc[t][i];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float v = red[0][t][tid / 16][tid % 16];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][t][tid / 16][tid % 16];
        out[t] = v;
    }
    __syncthreads();
}

template <int FMT>
__global__ __launch_bounds__(kThreads) void moe_gate_up_kernel(MoeLaunch p, MoeWs ws) {
    __shared__ Picked picked;
    __shared__ Partial red;
    int count = 0, reached;
    const int64_t e = __builtin_amdgcn_readfirstlane(
        pick_expert(ws.ids, p.tokens * p.top_k, blockIdx.y, picked, count, reached));
    if (e < 0) return;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int f0 = blockIdx.x * kUnits;
    const int kg = (p.dim + kGroup - 1) / kGroup, rg = (2 * p.hidden + kGroup - 1) / kGroup;
    const uint8_t* w[2];
    const float* s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {  // 16 rows share a tile of steps: hidden is a multiple of 16
        const int row = f0 + t * p.hidden;
        w[t] = p.w13 + (e * 2 * p.hidden + row + lane % 16) * p.dim + 16 * (lane / 16);
        s[t] = p.s13 + (e * rg + row / kGroup) * kg;
    }
    for (int c0 = 0; c0 < count; c0 += 16) {
        // lanes past the list repeat its last token; their results are dropped
        const int c = c0 + lane % 16 < count ? c0 + lane % 16 : count - 1;
        const uint16_t* const x[1] = {p.x + (int64_t)(picked.slot[c] / p.top_k) * p.dim +
                                      16 * (lane / 16)};
        v4f acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        tile_products<FMT, 1>(w, s, x, p.dim, wave, lane, acc);
        float v[2];
        join_waves(acc, red, v);
        if (c0 + tid / 16 < count) {
            const float h = v[0] / (1.0f + expf(-v[0])) * v[1];
            const int64_t o = (int64_t)picked.slot[c0 + tid / 16] * p.hidden + f0 + tid % 16;
            const uint16_t hi = f32_to_bf16(h);
            ws.h_hi[o] = hi;
            ws.h_lo[o] = f32_to_bf16(h - bf16_to_f32(hi));
        }
    }
}

template <int FMT>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeLaunch p, MoeWs ws) {
    __shared__ Picked picked;
    __shared__ Partial red;
    __shared__ uint32_t flag;
    int count = 0, reached;
    const int64_t e = __builtin_amdgcn_readfirstlane(
        pick_expert(ws.ids, p.tokens * p.top_k, blockIdx.y, picked, count, reached));
    if (e < 0) return;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int d0 = blockIdx.x * kRows;
    const int kg = (p.hidden + kGroup - 1) / kGroup, rg = (p.dim + kGroup - 1) / kGroup;
    const uint8_t* w[2];
    const float* s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        // dim is a multiple of 16: a second tile past it repeats the first
        const int row = d0 + 16 * t < p.dim ? d0 + 16 * t : d0;
        w[t] = p.w2 + (e * p.dim + row + lane % 16) * p.hidden + 16 * (lane / 16);
        s[t] = p.s2 + (e * rg + row / kGroup) * kg;
    }
    for (int c0 = 0; c0 < count; c0 += 16) {
        const int c = c0 + lane % 16 < count ? c0 + lane % 16 : count - 1;
        const int64_t at = (int64_t)picked.slot[c] * p.hidden + 16 * (lane / 16);
        const uint16_t* const h[2] = {ws.h_hi + at, ws.h_lo + at};
        v4f acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        tile_products<FMT, 2>(w, s, h, p.hidden, wave, lane, acc);
        float v[2];
        join_waves(acc, red, v);
        if (c0 + tid / 16 < count) {
            float* o = ws.part + (int64_t)picked.slot[c0 + tid / 16] * p.dim + d0 + tid % 16;
            store_dev(o, v[0]);
            if (d0 + 16 < p.dim) store_dev(o + 16, v[1]);
        }
    }
    // The last of the reached experts at these rows adds up every token's.
    if (!last_of(ws.down_count + blockIdx.x, reached, &flag)) return;
    const int cols = p.dim - d0 < kRows ? p.dim - d0 : kRows;
    for (int i = tid; i < p.tokens * kRows; i += kThreads) {
        const int t = i / kRows, d = i % kRows;
        if (d >= cols) continue;
        float y = 0.0f;
        for (int j = 0; j < p.top_k; ++j) {
            const int64_t slot = (int64_t)t * p.top_k + j;
            y = fmaf(ws.weights[slot], load_dev(ws.part + slot * p.dim + d0 + d), y);
        }
        p.out[(int64_t)t * p.dim + d0 + d] = f32_to_bf16(y);
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
    const dim3 up(p.hidden / kUnits, reach), down((p.dim + kRows - 1) / kRows, reach);
    if (p.fmt == 0) hipLaunchKernelGGL(moe_gate_up_kernel<0>, up, dim3(kThreads), 0, stream, p, ws);
    else hipLaunchKernelGGL(moe_gate_up_kernel<1>, up, dim3(kThreads), 0, stream, p, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (p.fmt == 0) hipLaunchKernelGGL(moe_down_kernel<0>, down, dim3(kThreads), 0, stream, p, ws);
    else hipLaunchKernelGGL(moe_down_kernel<1>, down, dim3(kThreads), 0, stream, p, ws);
    return hipGetLastError();
}

}  // namespace fp8lin
