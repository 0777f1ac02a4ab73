// Mixture-of-experts layer for a few tokens on tile-scaled fp8 weights:
//   l = x R^T;  the top_k experts e_j of each token (ties: lowest index);
//   w = softmax(l)[e_j], over their sum when asked;
//   y = sum_j w_j W2_e ( silu(G_e x) * (U_e x) ),  every weight = code * step.

#include "block.hpp"
#include "common.hpp"

namespace fp8lin {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxExperts = 512;

struct MoeWs {
    int32_t* ids;    // [tokens][top_k]
    float* weights;  // [tokens][top_k]
    float* h;        // [tokens * top_k][hidden]
};

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

MoeWs layout(void* ws, int64_t t, int64_t k, int64_t h, size_t* total) {
    uint8_t* p = static_cast<uint8_t*>(ws);
    MoeWs w;
    size_t at = 0;
    w.ids = reinterpret_cast<int32_t*>(p + at);
    at = up256(at + 4 * t * k);
    w.weights = reinterpret_cast<float*>(p + at);
    at = up256(at + 4 * t * k);
    w.h = reinterpret_cast<float*>(p + at);
    at = up256(at + 4 * t * k * h);
    *total = at;
    return w;
}

// One workgroup per token: logits in LDS, then wave 0 selects.
__global__ __launch_bounds__(kThreads) void moe_route_kernel(MoeLaunch p, MoeWs ws) {
    __shared__ float logit[kMaxExperts];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t t = blockIdx.x;
    const uint16_t* x = p.x + t * p.dim;
    for (int e = wave; e < p.experts; e += kThreads / kWave) {
        const uint16_t* r = p.router + (int64_t)e * p.dim;
        float s = 0.0f;
        for (int d = lane; d < p.dim; d += kWave) s = fmaf(bf16_to_f32(x[d]), bf16_to_f32(r[d]), s);
        s = wave_sum(s);
        if (lane == 0) logit[e] = s;
    }
    __syncthreads();
    if (wave != 0) return;
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

__device__ __forceinline__ float code_value(int fmt, uint8_t c) {
    return fmt ? dec8<1, 0>(c) : dec8<0, 0>(c);
}

// One wave per (token's chosen expert, hidden unit): both dot products.
__global__ __launch_bounds__(kThreads) void moe_gate_up_kernel(MoeLaunch p, MoeWs ws) {
    const int lane = threadIdx.x % kWave;
    const int f = blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
    const int64_t slot = blockIdx.y;
    if (f >= p.hidden) return;
    const int64_t e = ws.ids[slot];
    const uint16_t* x = p.x + slot / p.top_k * p.dim;
    const int kg = (p.dim + kGroup - 1) / kGroup, rg = (2 * p.hidden + kGroup - 1) / kGroup;
    float acc[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int row = f + u * p.hidden;
        const uint8_t* w = p.w13 + (e * 2 * p.hidden + row) * p.dim;
        const float* s = p.s13 + (e * rg + row / kGroup) * kg;
        float a = 0.0f;
        for (int d = lane; d < p.dim; d += kWave)
            a = fmaf(code_value(p.fmt, w[d]) * s[d / kGroup], bf16_to_f32(x[d]), a);
        acc[u] = wave_sum(a);
    }
    if (lane == 0) ws.h[slot * p.hidden + f] = acc[0] / (1.0f + expf(-acc[0])) * acc[1];
}

// One wave per (token, output): the weighted sum over its experts.
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeLaunch p, MoeWs ws) {
    const int lane = threadIdx.x % kWave;
    const int d = blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
    const int64_t t = blockIdx.y;
    if (d >= p.dim) return;
    const int kg = (p.hidden + kGroup - 1) / kGroup, rg = (p.dim + kGroup - 1) / kGroup;
    float y = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
        const int64_t slot = t * p.top_k + j;
        const int64_t e = ws.ids[slot];
        const uint8_t* w = p.w2 + (e * p.dim + d) * p.hidden;
        const float* s = p.s2 + (e * rg + d / kGroup) * kg;
        float a = 0.0f;
        for (int f = lane; f < p.hidden; f += kWave)
            a = fmaf(code_value(p.fmt, w[f]) * s[f / kGroup], ws.h[slot * p.hidden + f], a);
        y = fmaf(ws.weights[slot], wave_sum(a), y);
    }
    if (lane == 0) p.out[t * p.dim + d] = f32_to_bf16(y);
}

}  // namespace

size_t moe_workspace(int64_t tokens, int64_t, int64_t top_k, int64_t, int64_t hidden) {
    size_t total;
    layout(nullptr, tokens, top_k, hidden, &total);
    return total;
}

hipError_t launch_moe(const MoeLaunch& p, hipStream_t stream) {
    size_t total;
    const MoeWs ws = layout(p.ws, p.tokens, p.top_k, p.hidden, &total);
    constexpr int kPer = kThreads / kWave;
    hipLaunchKernelGGL(moe_route_kernel, dim3(p.tokens), dim3(kThreads), 0, stream, p, ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_gate_up_kernel, dim3((p.hidden + kPer - 1) / kPer, p.tokens * p.top_k),
                       dim3(kThreads), 0, stream, p, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(moe_down_kernel, dim3((p.dim + kPer - 1) / kPer, p.tokens), dim3(kThreads),
                       0, stream, p, ws);
    return hipGetLastError();
}

}  // namespace fp8lin
