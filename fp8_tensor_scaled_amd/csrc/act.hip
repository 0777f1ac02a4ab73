// Activations, gated or not, that keep their input in 8 bits.
//
// Forward: y = a(x), or a(gate) * up, from the input as it is; its codes and
// steps (fp8_quantize_block's row grouping, each half of a gated row for
// itself) from the same read.  Backward: x' = code * step, dx = g a'(x').
//
// Sixteen lanes hold a group of 128 columns, eight each (and the same eight of
// the other half): a step's maximum is theirs alone, 16-byte loads and stores
// of a 2-byte type, no LDS.  A workgroup works on one set of groups: two rows a
// lane took 4 % longer at 16384 x 4096, gated bf16.
//
// Bandwidth bound: forward 16384 x 4096 gated bf16 with its checkpoint 77 us
// (541 MB, 7.0 TB/s), backward 89 (6.1 TB/s), calls in a row; 84 and 96 where each
// ends before the next begins.  The checkpoint, which is read much later, is
// written past the caches, y and dx, which the next operator reads, through
// them (see written_early for smaller ones): with a block quantize of the output
// behind it, forward 125 us and backward 167; with all written past the caches 135
// and 173, none 132 and 168.

#include "expert_block.hpp"
#include "rows.hpp"

namespace fp8lin {

namespace {

constexpr int kT = 256, kPlaces = kT / 16;  // groups of a workgroup at a time
constexpr int kMostRowBlocks = 65535;       // a grid's second dimension

enum Act : int { kSilu = 0, kGelu = 1, kGeluTanh = 2 };

// exp(-u) by the hardware's exponential: the product and its constant are rounded,
// so off by 1.3 |u| + 2 half steps of fp32.
__device__ __forceinline__ float exp_minus(float u) {
    return __builtin_amdgcn_exp2f(u * -1.4426950408889634f);
}

// 1 / (1 + exp(-u)) and what is left of 1.  For a 2-byte type by the hardware's
// exponential and reciprocal: off by 1.3 |u| + 5 half steps of fp32, of which the type's
// own half step has 2^13 (fp16) or 2^16.  For fp32 a whole exponential, of -|u|, so
// that it ends nowhere before the result does, and a whole division: either within
// 5 half steps.  (silu on [-20, 20] is off by up to 3.7 with this form, by 16.7 with
// the short one; 8192 x 4096 gated with its checkpoint takes 85 us forwards and 93
// backwards, with the short one 83 and 91: the memory's time, 5.5 and 5.1 TB/s.)
struct Logistic {
    float p, rest;
};
template <int IN>
__device__ __forceinline__ Logistic logistic(float u) {
    if constexpr (IN == kInF32) {
        const float e = expf(-fabsf(u));
        const float large = 1.0f / (1.0f + e), small = e * large;
        return {u < 0.0f ? small : large, u < 0.0f ? large : small};
    } else {
        const float p = __builtin_amdgcn_rcpf(1.0f + exp_minus(u));
        return {p, 1.0f - p};
    }
}

// The standard normal distribution P and its density at v.  With a = |v|,
// P(-a) = exp(-a^2 / 2) t Q(t) / 2, t = 1 / (1 + 0.35 a / sqrt 2), where t Q(t)
// stands for erfc(a / sqrt 2) exp(a^2 / 2): Q of degree 9, fitted to 64-bit
// values on 0 <= a <= 20 with least squares reweighted to a level error, which
// is 1.1e-8 of the value (6 half steps of fp32 as computed).  One exponential
// serves both, and there is no branch (16384 x 4096 gated with its checkpoint:
// forward 85 us, silu 79; with the library's erfc, exponential and divisions 130).
struct Normal {
    float p, density;
};
__device__ __forceinline__ Normal normal(float v) {
    const float a = fabsf(v);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.24748737f, a, 1.0f));
    float q = 0.04184477f;
    q = fmaf(q, t, -0.1779024601f);
    q = fmaf(q, t, 0.2267737091f);
    q = fmaf(q, t, -0.08914090693f);
    q = fmaf(q, t, 0.1390236169f);
    q = fmaf(q, t, 0.1176004633f);
    q = fmaf(q, t, 0.1612146497f);
    q = fmaf(q, t, 0.1857084185f);
    q = fmaf(q, t, 0.1974081546f);
    q = fmaf(q, t, 0.1974695921f);
    const float e = exp_minus(0.5f * v * v);
    const float below = 0.5f * e * (t * q);
    return {v >= 0.0f ? 1.0f - below : below, 0.3989422804f * e};
}

// v P(v) and its slope P(v) + v P'(v): P is 1 / (1 + exp(-v)) (silu), the
// standard normal distribution (gelu) or 1 / (1 + exp(-2u(v))) (gelu_tanh).
template <int IN, int ACT>
__device__ __forceinline__ float value_of(float v) {
    if constexpr (ACT == kSilu) return v * logistic<IN>(v).p;
    if constexpr (ACT == kGelu) return v * normal(v).p;
    return v * logistic<IN>(1.5957691216f * v * fmaf(0.044715f * v, v, 1.0f)).p;
}

struct ValueSlope {
    float value, slope;
};
template <int IN, int ACT>
__device__ __forceinline__ ValueSlope value_slope(float v) {
    float p, d;  // P, P'
    if constexpr (ACT == kSilu) {
        const Logistic l = logistic<IN>(v);
        p = l.p;
        d = p * l.rest;
    } else if constexpr (ACT == kGelu) {
        const Normal n = normal(v);
        p = n.p;
        d = n.density;
    } else {
        const Logistic l = logistic<IN>(1.5957691216f * v * fmaf(0.044715f * v, v, 1.0f));
        p = l.p;
        // (v^2 bounded: p (1 - p) is 0 long before, and must stay it)
        d = p * l.rest * 1.5957691216f * fmaf(0.134145f, fminf(v * v, 1e30f), 1.0f);
    }
    return {v * p, fmaf(v, d, p)};
}

// A workgroup's groups: 2^shift of them side by side (the most, up to
// kPlaces, that divide a row's groups, so that none is left over), on
// kPlaces >> shift rows.
struct Places {
    int shift;
    int64_t groups;
    __device__ int64_t column_group() const {
        return ((int64_t)blockIdx.x << shift) + ((threadIdx.x / 16) & ((1 << shift) - 1));
    }
    __device__ int64_t first_row() const {
        return (int64_t)blockIdx.y * (kPlaces >> shift) + (threadIdx.x / 16 >> shift);
    }
    __device__ int64_t rows_on() const { return (int64_t)gridDim.y * (kPlaces >> shift); }
};

template <int IN, int ACT, bool GATED, bool KEEP>
__global__ __launch_bounds__(kT) void act_fwd_kernel(ActLaunch p, Places at) {
    constexpr int kHalves = GATED ? 2 : 1;
    const int64_t cg = at.column_group();
    const int64_t c = cg * kGroup + 8 * (threadIdx.x % 16);
    // (the 16 lanes of a group are in the loop together)
    for (int64_t r = at.first_row(); r < p.rows; r += at.rows_on()) {
        const void* x = row_at<IN>(p.in, r, p.ld);
        Raw8<IN> raw[kHalves];
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
            raw[h] = load_row8<IN, true>(row_at<IN>(x, h, p.cols), c, p.cols);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[j] = value_of<IN, ACT>(raw[0][j]);
            if constexpr (GATED) y[j] *= raw[1][j];
        }
        store_row8<IN>(row_at<IN>(p.out, r, p.cols), c, p.cols, y, p.early);
        if constexpr (KEEP) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                float v[8];
                raw[h].values(v);
                const Codes8 q = group_codes(p.fmt, v, p.rmargin);
                uint8_t* row = p.x8 + (r * kHalves + h) * p.cols;
                if (c + 8 <= p.cols) {
                    typedef uint32_t AnyVec2 __attribute__((ext_vector_type(2), aligned(1)));
                    __builtin_nontemporal_store(AnyVec2{q.lo, q.hi},
                                                reinterpret_cast<AnyVec2*>(row + c));
                } else {
                    store8(row, 0, c, p.cols, 0, q.lo, q.hi);
                }
                if (threadIdx.x % 16 == 0) p.steps[(r * kHalves + h) * at.groups + cg] = q.step;
            }
        }
    }
}

// Codes of columns c .. c + 7, zeros from `cols` on.
__device__ __forceinline__ uint2 load_codes(const uint8_t* row, int64_t c, int64_t cols) {
    uint2 w = make_uint2(0, 0);
    if (c + 8 <= cols) {
        __builtin_memcpy(&w, row + c, 8);
        return w;
    }
    uint64_t one = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j < cols) one |= (uint64_t)row[c + j] << (8 * j);
    return make_uint2((uint32_t)one, (uint32_t)(one >> 32));
}

template <int FMT>
__device__ __forceinline__ void decode8(uint2 w, float step, float (&v)[8]) {
    v[0] = dec8<FMT, 0>(w.x) * step;
    v[1] = dec8<FMT, 1>(w.x) * step;
    v[2] = dec8<FMT, 2>(w.x) * step;
    v[3] = dec8<FMT, 3>(w.x) * step;
    v[4] = dec8<FMT, 0>(w.y) * step;
    v[5] = dec8<FMT, 1>(w.y) * step;
    v[6] = dec8<FMT, 2>(w.y) * step;
    v[7] = dec8<FMT, 3>(w.y) * step;
}

template <int IN, int ACT, bool GATED>
__global__ __launch_bounds__(kT) void act_bwd_kernel(ActLaunch p, Places at) {
    constexpr int kHalves = GATED ? 2 : 1;
    const int64_t cg = at.column_group();
    const int64_t c = cg * kGroup + 8 * (threadIdx.x % 16);
    for (int64_t r = at.first_row(); r < p.rows; r += at.rows_on()) {
        const Raw8<IN> g = load_row8<IN, true>(row_at<IN>(p.in, r, p.ld), c, p.cols);
        float v[kHalves][8], d[8], e[8];
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const uint2 w = load_codes(p.x8 + (r * kHalves + h) * p.cols, c, p.cols);
            const float step = p.steps[(r * kHalves + h) * at.groups + cg];
            if (p.fmt)
                decode8<1>(w, step, v[h]);
            else
                decode8<0>(w, step, v[h]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const ValueSlope a = value_slope<IN, ACT>(v[0][j]);
            if constexpr (GATED) {
                d[j] = g[j] * v[1][j] * a.slope;
                e[j] = g[j] * a.value;
            } else {
                d[j] = g[j] * a.slope;
            }
        }
        void* dx = row_at<IN>(p.out, r * kHalves, p.cols);
        store_row8<IN>(dx, c, p.cols, d, p.early);
        if constexpr (GATED) store_row8<IN>(row_at<IN>(dx, 1, p.cols), c, p.cols, e, p.early);
    }
}

struct Launch {
    dim3 grid;
    Places at;
};
Launch launch_of(const ActLaunch& q) {
    Launch l;
    l.at.groups = groups_of(q.cols);
    l.at.shift = 0;
    while ((1 << l.at.shift) < kPlaces && (l.at.groups >> l.at.shift) % 2 == 0) ++l.at.shift;
    const int64_t rows = kPlaces >> l.at.shift;
    const int64_t blocks = (q.rows + rows - 1) / rows;
    l.grid = dim3((unsigned)(l.at.groups >> l.at.shift),
                  (unsigned)(blocks < kMostRowBlocks ? blocks : kMostRowBlocks));
    return l;
}

template <int IN, int ACT, bool GATED, bool BWD>
hipError_t launch_one(const ActLaunch& q, hipStream_t stream) {
    const Launch l = launch_of(q);
    if constexpr (BWD)
        hipLaunchKernelGGL((act_bwd_kernel<IN, ACT, GATED>), l.grid, dim3(kT), 0, stream, q, l.at);
    else if (q.x8)
        hipLaunchKernelGGL((act_fwd_kernel<IN, ACT, GATED, true>), l.grid, dim3(kT), 0, stream, q,
                           l.at);
    else
        hipLaunchKernelGGL((act_fwd_kernel<IN, ACT, GATED, false>), l.grid, dim3(kT), 0, stream, q,
                           l.at);
    return hipGetLastError();
}
template <int IN, int ACT, bool BWD>
hipError_t launch_gated(const ActLaunch& q, hipStream_t stream) {
    return q.gated ? launch_one<IN, ACT, true, BWD>(q, stream)
                   : launch_one<IN, ACT, false, BWD>(q, stream);
}
template <int IN, bool BWD>
hipError_t launch_act(const ActLaunch& q, hipStream_t stream) {
    switch (q.act) {
        case kSilu: return launch_gated<IN, kSilu, BWD>(q, stream);
        case kGelu: return launch_gated<IN, kGelu, BWD>(q, stream);
        default: return launch_gated<IN, kGeluTanh, BWD>(q, stream);
    }
}
template <bool BWD>
hipError_t launch_type(const ActLaunch& q, hipStream_t stream) {
    if (q.type == kInBf16) return launch_act<kInBf16, BWD>(q, stream);
    return q.type == kInF16 ? launch_act<kInF16, BWD>(q, stream)
                            : launch_act<kInF32, BWD>(q, stream);
}

}  // namespace

hipError_t launch_act_fwd(const ActLaunch& of, hipStream_t stream) {
    ActLaunch q = of;
    const int64_t n = q.rows * q.cols, size = size_of(q.type);
    q.early = written_early(n * size + (q.x8 ? n * (1 + q.gated) : 0), q.cols * size);
    return launch_type<false>(q, stream);
}
hipError_t launch_act_bwd(const ActLaunch& of, hipStream_t stream) {
    ActLaunch q = of;
    const int64_t size = size_of(q.type);
    q.early = written_early(q.rows * q.cols * (1 + q.gated) * size, q.cols * size);
    return launch_type<true>(q, stream);
}

}  // namespace fp8lin
