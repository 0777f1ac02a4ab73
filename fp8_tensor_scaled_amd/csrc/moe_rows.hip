// Tokens into the experts' order and back.
//     dispatch      rows[slot(t, j)] = x[t]
//     combine       out[t] = sum_j w(t, j) rows[slot(t, j)]
//     its backward  drows[slot(t, j)] = w(t, j) g[t],   dw(t, j) = <g[t], rows[slot(t, j)]>
// All go by token: a token's row is read (or written) once for its top_k
// rows, whatever their order.  A pair of no expert has a slot from `total` on:
// its row gets zeros and counts for nothing.
//
// Bandwidth bound: a lane holds 16 bytes of a token (eight columns of a 2-byte
// type, four of fp32), a wave 1 KB of it, or, where tokens are narrower, 16 or 32
// of its lanes one each.  It has the loads of all choices under way before it
// uses the first, so the number of choices is a template argument (the next of
// 1, 2, 4, 8, 16: one of 3, 5, 6 or 7 of its own gains nothing there and in combine;
// combine's backward with the next / its own, bf16: 2048 tokens of 1024, 3 choices
// 7.0 / 6.8 us, 5 11.5 / 10.9, 6 13.1 / 12.5, 7 13.9 / 13.7; 16384 of 2048 94 / 93,
// 149 / 149, 176 / 176, 207 / 208).  Rows are read once: past the caches (combine 102
// us, 119 without, at 131072 rows of 2048 bf16).  They are written through them, for
// the next operator: dispatch of that size takes 111 us so and 102 past the caches,
// but with a block quantize of its rows behind it 249 and 277.

#include "expert_block.hpp"
#include "rows.hpp"

namespace fp8lin {

namespace {

constexpr int kT = 256;

// 16 bytes of a row: columns c .. c + kN - 1, zeros behind the row's end.
template <int IN>
struct Vec {
    using V = typename Elem<IN>::T;
    static constexpr int kN = 16 / (int)sizeof(V);
    AnyVec4 w;
    __device__ float operator[](int j) const {
        if constexpr (IN == kInF32) return __uint_as_float(w[j]);
        if constexpr (IN == kInBf16) return j % 2 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
        return Elem<IN>::f((V)(j % 2 ? w[j / 2] >> 16 : w[j / 2]));
    }
};
template <int IN, bool NT>
__device__ __forceinline__ Vec<IN> load_vec(const void* row, int64_t c, int64_t cols) {
    using V = typename Elem<IN>::T;
    constexpr int N = Vec<IN>::kN;
    const V* src = static_cast<const V*>(row) + c;
    Vec<IN> r;
    if (c + N <= cols) {
        if constexpr (NT)
            r.w = __builtin_nontemporal_load(reinterpret_cast<const AnyVec4*>(src));
        else
            r.w = *reinterpret_cast<const AnyVec4*>(src);
    } else {
        V one[N];
#pragma unroll
        for (int j = 0; j < N; ++j) one[j] = c + j < cols ? src[j] : V(0);
        __builtin_memcpy(&r.w, one, sizeof one);
    }
    return r;
}
template <int IN>
__device__ __forceinline__ Vec<IN> pack_vec(const float (&v)[Vec<IN>::kN]) {
    Vec<IN> r;
    if constexpr (IN == kInF32) {
        __builtin_memcpy(&r.w, v, sizeof r.w);
    } else {
        const Pack<IN> p(v);
        __builtin_memcpy(&r.w, p.w, sizeof r.w);
    }
    return r;
}
template <int IN>
__device__ __forceinline__ void store_vec(void* row, int64_t c, int64_t cols, const Vec<IN>& v,
                                          bool early) {
    using V = typename Elem<IN>::T;
    constexpr int N = Vec<IN>::kN;
    V* dst = static_cast<V*>(row) + c;
    if (c + N <= cols) {
        store16(reinterpret_cast<AnyVec4*>(dst), v.w, early);
    } else {
        V one[N];
        __builtin_memcpy(one, &v.w, sizeof one);
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (c + j < cols) dst[j] = one[j];
    }
}

// A token's choices: where its rows are, and which of them an expert has.
template <int K>
struct Choices {
    int slot[K];
    uint32_t inside = 0;  // bit j: a row of the buffer
    uint32_t expert = 0;  // bit j: ... that has an expert
    __device__ Choices(const MoeRowsLaunch& p, int64_t t, int total) {
        const int rows = (int)(p.tokens * p.top_k);
#pragma unroll
        for (int j = 0; j < K; ++j)
            slot[j] = j < p.top_k ? p.slots[t * p.top_k + j] : -1;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            inside |= (uint32_t)(slot[j] >= 0 && slot[j] < rows) << j;
            expert |= (uint32_t)(slot[j] >= 0 && slot[j] < rows && slot[j] < total) << j;
        }
    }
};

// The piece of a token that LANES neighbouring lanes hold: token `t` (past the
// last where there is none) and this lane's first column.  A whole wave's
// token is kept as a scalar, and so are its slots.
template <int IN, int LANES>
struct Piece {
    int64_t t, c;
    __device__ explicit Piece(int pieces) {
        const int lane = threadIdx.x % LANES;
        int place = threadIdx.x / LANES;
        if constexpr (LANES == kWave) place = __builtin_amdgcn_readfirstlane(place);
        const int64_t id = workgroup_id() * (kT / LANES) + place;
        t = id / pieces;
        c = (id % pieces * LANES + lane) * Vec<IN>::kN;
    }
};

template <int IN, int K, int LANES>
__global__ __launch_bounds__(kT) void dispatch_kernel(MoeRowsLaunch p, int pieces) {
    const Piece<IN, LANES> at(pieces);
    if (at.t >= p.tokens) return;
    const Choices<K> to(p, at.t, *p.total);
    if (at.c >= p.dim) return;
    const Vec<IN> v = load_vec<IN, false>(row_at<IN>(p.in, at.t, p.ld), at.c, p.dim);
    const Vec<IN> zero = {};
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (!(to.inside >> j & 1)) continue;
        store_vec<IN>(row_at<IN>(p.out, to.slot[j], p.dim), at.c, p.dim,
                      to.expert >> j & 1 ? v : zero, p.early);
    }
}

template <int IN, int K, int LANES>
__global__ __launch_bounds__(kT) void combine_kernel(MoeRowsLaunch p, int pieces) {
    constexpr int N = Vec<IN>::kN;
    const Piece<IN, LANES> at(pieces);
    const int64_t t = at.t, c = at.c;
    if (t >= p.tokens) return;
    const Choices<K> from(p, t, *p.total);
    if (c >= p.dim) return;
    Vec<IN> raw[K];
    float w[K], sum[N] = {};
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (!(from.expert >> j & 1)) continue;
        raw[j] = load_vec<IN, true>(row_at<IN>(p.in, from.slot[j], p.dim), c, p.dim);
        w[j] = p.weights ? p.weights[t * p.top_k + j] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (!(from.expert >> j & 1)) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] = fmaf(w[j], raw[j][i], sum[i]);
    }
    store_vec<IN>(row_at<IN>(p.out, t, p.dim), c, p.dim, pack_vec<IN>(sum), p.early);
}

// LANES lanes hold a token, 16 LANES bytes at a time.
template <int IN, int K, int LANES>
__global__ __launch_bounds__(kT) void combine_bwd_kernel(MoeRowsLaunch p) {
    constexpr int N = Vec<IN>::kN;
    __shared__ float red[kT / 16][K];
    int place = threadIdx.x / LANES;
    if constexpr (LANES >= kWave) place = __builtin_amdgcn_readfirstlane(place);
    const int lane = threadIdx.x % LANES;
    const int64_t t = workgroup_id() * (kT / LANES) + place;
    const bool mine = t < p.tokens;
    float dot[K] = {};
    if (mine) {
        const Choices<K> at(p, t, *p.total);
        const void* g = row_at<IN>(p.in, t, p.ld);
        for (int64_t c = N * lane; c < p.dim; c += N * LANES) {
            const Vec<IN> gv = load_vec<IN, false>(g, c, p.dim);
            Vec<IN> y[K];
            if (p.dweights) {
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (at.expert >> j & 1)
                        y[j] = load_vec<IN, true>(row_at<IN>(p.rows, at.slot[j], p.dim), c, p.dim);
            }
            if (p.out) {
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    if (!(at.inside >> j & 1)) continue;
                    float d[N] = {};
                    if (at.expert >> j & 1) {
                        const float w = p.weights[t * p.top_k + j];
#pragma unroll
                        for (int i = 0; i < N; ++i) d[i] = w * gv[i];
                    }
                    store_vec<IN>(row_at<IN>(p.out, at.slot[j], p.dim), c, p.dim, pack_vec<IN>(d),
                                  p.early);
                }
            }
            if (p.dweights) {
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    if (!(at.expert >> j & 1)) continue;
#pragma unroll
                    for (int i = 0; i < N; ++i) dot[j] = fmaf(gv[i], y[j][i], dot[j]);
                }
            }
        }
    }
    if (!p.dweights) return;
    // sums over 16 lanes or a wave, then over a token's parts of that size
    constexpr int kOf = LANES < kWave ? 16 : kWave, kParts = LANES / kOf;
#pragma unroll
    for (int j = 0; j < K; ++j) dot[j] = sum_lanes<kOf>(dot[j]);
    const int part = threadIdx.x / kOf;
    if (threadIdx.x % kOf == 0) {
#pragma unroll
        for (int j = 0; j < K; ++j) red[part][j] = dot[j];
    }
    __syncthreads();
    if (!mine || lane >= p.top_k) return;
    const int first = part / kParts * kParts;
    float s = red[first][lane];
#pragma unroll
    for (int w = 1; w < kParts; ++w) s += red[first + w][lane];
    p.dweights[t * p.top_k + lane] = s;
}

// fn(type, choices) as compile-time numbers.
template <int N>
struct Number {
    static constexpr int value = N;
};
template <class Fn>
hipError_t with_choices(const MoeRowsLaunch& q, Fn fn) {
    if (q.top_k == 1) return fn(Number<1>{});
    if (q.top_k == 2) return fn(Number<2>{});
    if (q.top_k <= 4) return fn(Number<4>{});
    if (q.top_k <= 8) return fn(Number<8>{});
    return fn(Number<16>{});
}
template <class Fn>
hipError_t with_type(const MoeRowsLaunch& q, Fn fn) {
    const auto of_type = [&](auto in) {
        return with_choices(q, [&](auto k) {
            fn(in, k);
            return hipGetLastError();
        });
    };
    if (q.type == kInBf16) return of_type(Number<kInBf16>{});
    return q.type == kInF16 ? of_type(Number<kInF16>{}) : of_type(Number<kInF32>{});
}

// fn(type, choices, lanes) for a kernel whose lane groups hold pieces of a token.
template <class Fn>
hipError_t with_lanes(const MoeRowsLaunch& q, Fn fn) {
    return with_type(q, [&](auto in, auto k) {
        constexpr int N = Vec<decltype(in)::value>::kN;
        if (q.dim <= N * 16)
            fn(in, k, Number<16>{});
        else if (q.dim <= N * 32)
            fn(in, k, Number<32>{});
        else
            fn(in, k, Number<64>{});
    });
}

template <int IN, int LANES>
int pieces_of(const MoeRowsLaunch& q) {
    constexpr int of_piece = Vec<IN>::kN * LANES;
    return (int)((q.dim + of_piece - 1) / of_piece);
}
// Workgroups of kT lanes, LANES for each of `items`.
template <int LANES>
dim3 lanes_grid(int64_t items) {
    return grid_of((items + kT / LANES - 1) / (kT / LANES));
}

// For `rows` rows a token written.
bool early_of(const MoeRowsLaunch& q, int rows) {
    const int64_t row = q.dim * size_of(q.type);
    return written_early(q.tokens * rows * row, row);
}

}  // namespace

hipError_t launch_moe_dispatch(const MoeRowsLaunch& of, hipStream_t stream) {
    MoeRowsLaunch q = of;
    q.early = early_of(q, q.top_k);
    return with_lanes(q, [&](auto in, auto k, auto lanes) {
        constexpr int IN = decltype(in)::value, L = decltype(lanes)::value;
        const int pieces = pieces_of<IN, L>(q);
        hipLaunchKernelGGL((dispatch_kernel<IN, decltype(k)::value, L>),
                           lanes_grid<L>(q.tokens * pieces), dim3(kT), 0, stream, q, pieces);
    });
}

hipError_t launch_moe_combine(const MoeRowsLaunch& of, hipStream_t stream) {
    MoeRowsLaunch q = of;
    q.early = early_of(q, 1);
    return with_lanes(q, [&](auto in, auto k, auto lanes) {
        constexpr int IN = decltype(in)::value, L = decltype(lanes)::value;
        const int pieces = pieces_of<IN, L>(q);
        hipLaunchKernelGGL((combine_kernel<IN, decltype(k)::value, L>),
                           lanes_grid<L>(q.tokens * pieces), dim3(kT), 0, stream, q, pieces);
    });
}

hipError_t launch_moe_combine_bwd(const MoeRowsLaunch& of, hipStream_t stream) {
    MoeRowsLaunch q = of;
    q.early = early_of(q, q.top_k);
    return with_lanes(q, [&](auto in, auto k, auto lanes) {
        constexpr int IN = decltype(in)::value, K = decltype(k)::value;
        constexpr int L = decltype(lanes)::value;
        constexpr int64_t wave = Vec<IN>::kN * kWave;  // columns
        if constexpr (L == kWave) {
            if (q.dim > 2 * wave) {
                hipLaunchKernelGGL((combine_bwd_kernel<IN, K, 4 * kWave>),
                                   lanes_grid<4 * kWave>(q.tokens), dim3(kT), 0, stream, q);
                return;
            }
            if (q.dim > wave) {
                hipLaunchKernelGGL((combine_bwd_kernel<IN, K, 2 * kWave>),
                                   lanes_grid<2 * kWave>(q.tokens), dim3(kT), 0, stream, q);
                return;
            }
        }
        hipLaunchKernelGGL((combine_bwd_kernel<IN, K, L>), lanes_grid<L>(q.tokens), dim3(kT), 0,
                           stream, q);
    });
}

}  // namespace fp8lin
