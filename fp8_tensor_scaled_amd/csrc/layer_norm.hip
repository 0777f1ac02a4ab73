// Layer norm over the last dimension and its gradients.
//     y  = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean of (x - mean)^2 + eps)
//     h  = (x - mean) rstd,  v = g w
//     dx = rstd (v - mean v - h mean(v h)),   dw = sum g h,   db = sum g
// The variance is the mean of squared distances from the mean, not a
// difference of two large sums.
//
// Bandwidth bound when large: 16384 x 4096 bf16 forward 50 us (268 MB, 5.4 TB/s),
// backward 76 (403 MB and 8 MB of partial sums written and read, 5.5 TB/s); a
// large copy reaches 5.0 to 5.2.  fp32: 102 and 153 us, 5.3 TB/s both.  Small ones are
// bound by a row's chain (load, sums, store): 2048 x 1024 forward 4.0 us, backward
// 8.3.  (Calls in a row; traced one by one 53, 71 + 5 and 5.2, 5.7 + 3.2.)
//
// A row is held in registers up to 16384 columns, by 8 to 32 lanes up to 256
// columns, by a wave up to 1024, by several waves from there on; the columns' sums of the
// backward stay in registers too, over all rows of a workgroup, and meet in LDS at
// its end.  So x and g are read once.  From 8193 columns on not all of the backward's
// sums fit: the compiler puts 124 bytes a lane into memory for fp32 (204 where the
// width is no multiple of 8) and 64 for the 2-byte types of such a width, none for
// them otherwise.  4096 x 16384 forward / backward: bf16 60 / 84 us, 4.5 / 4.8 TB/s;
// of 16383 columns 96 / 138, 2.8 / 2.9; fp32 115 / 219, 4.7 / 3.7; of 16383 129 /
// 252, 4.2 / 3.2.

#include "expert_block.hpp"
#include "rows.hpp"

namespace fp8lin {

namespace {

constexpr int kT = 1024;  // lanes of a workgroup for rows of any length

// The workgroup's sum, in every lane.
template <int T>
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = wave_sum(v);
    __syncthreads();
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int w = 1; w < T / kWave; ++w) s += red[w];
    return s;
}

// Columns c .. c + 7 of a parameter (`fill` without one).
template <int IN, bool WHOLE = false>
__device__ __forceinline__ void load_param(const void* p, bool f32, int64_t c, int64_t cols,
                                           float fill, float (&v)[8]) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fill;
    } else if (f32) {
        load_row8<kInF32, false, WHOLE>(p, c, cols).values(v);
    } else {
        load_row8<IN, false, WHOLE>(p, c, cols).values(v);
    }
}

// ---- rows held in registers ----------------------------------------------
//
// LANES neighbouring lanes hold a row, V times eight columns each (lane l:
// columns 8 (l + LANES i) .. + 7).  A workgroup of T lanes works on T / LANES rows
// at a time and goes on to the rows a grid further, whose loads are under way
// while it finishes the ones it has; the parameters stay in registers.  512 lanes
// a workgroup: backward 16384 x 4096 bf16 73 us, with 256 and two on a CU 77 (twice
// as many partial sums).

// WHOLE: the row's length is a multiple of 8.
template <int LANES, int V, bool WHOLE>
struct Shape {
    static constexpr int kLanes = LANES, kV = V;
    static constexpr bool kWhole = WHOLE;
    static constexpr bool kTwice = V == 4;  // see bwd_rows
    static constexpr int kT = 512;
    static constexpr int kRows = kT / LANES;  // rows at a time
};

// Sums over a row's lanes, in every lane, N at a time.  `red` is
// [2][N][T / kWave] floats of LDS; `turn` alternates from call to call, so that
// one barrier a call is enough: a half is written again only two calls on,
// past a barrier that every wave reaches after it has read it.
template <class S, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int turn) {
    constexpr int kOfWave = S::kLanes < kWave ? S::kLanes : kWave;
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = sum_lanes<kOfWave>(v[n]);
    if constexpr (S::kLanes > kWave) {
        constexpr int kWaves = S::kT / kWave, kOf = S::kLanes / kWave;
        float* mine = red + turn * N * kWaves;
        const int wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) mine[n * kWaves + wave] = v[n];
        }
        __syncthreads();
        const int first = wave / kOf * kOf;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = mine[n * kWaves + first];
#pragma unroll
            for (int w = 1; w < kOf; ++w) s += mine[n * kWaves + first + w];
            v[n] = s;
        }
    }
}

// Raw columns of a row, `V` times eight.
template <int IN, class S>
struct RowRaw {
    Raw8<IN> v[S::kV];
    __device__ void load(const void* row, int l, int64_t cols) {
#pragma unroll
        for (int i = 0; i < S::kV; ++i)
            v[i] = load_row8<IN, true, S::kWhole>(row, 8 * (l + S::kLanes * i), cols);
    }
    // Makes the compiler take the values for new ones, and so compute again what
    // it would have kept.
    __device__ void forget() {
#pragma unroll
        for (int i = 0; i < S::kV; ++i) {
#pragma unroll
            for (int z = 0; z < Raw8<IN>::kVecs; ++z) asm("" : "+v"(v[i].v[z]));
        }
    }
};

template <int IN, class S, bool CODES>
__global__ __launch_bounds__(S::kT) void norm_fwd_rows_kernel(NormFwdLaunch p) {
    constexpr int V = S::kV;
    __shared__ float red[2 * (S::kT / kWave)];
    const int l = threadIdx.x % S::kLanes;
    const int64_t step = (int64_t)gridDim.x * S::kRows;
    const int64_t r0 = (int64_t)blockIdx.x * S::kRows + threadIdx.x / S::kLanes;
    const float n = (float)p.cols;
    float w[V][8], b[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load_param<IN, S::kWhole>(p.weight, p.w_f32, 8 * (l + S::kLanes * i), p.cols, 1.0f, w[i]);
        load_param<IN, S::kWhole>(p.bias, p.w_f32, 8 * (l + S::kLanes * i), p.cols, 0.0f, b[i]);
    }
    RowRaw<IN, S> next;
    if (r0 < p.rows) next.load(row_at<IN>(p.x, r0, p.ldx), l, p.cols);
    // (every lane of the workgroup takes part in every turn: the sums' barriers)
    const int64_t first = (int64_t)blockIdx.x * S::kRows;
    for (int64_t at = first; at < p.rows; at += step) {
        const int64_t r = at + threadIdx.x / S::kLanes;
        const bool mine = r < p.rows;
        const RowRaw<IN, S> raw = next;
        if (r + step < p.rows) next.load(row_at<IN>(p.x, r + step, p.ldx), l, p.cols);
        float v[V][8], s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            raw.v[i].values(v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += v[i][j];
        }
        row_sums<S, 1>(s, red, 0);
        const float mean = s[0] / n;
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t c = 8 * (l + S::kLanes * i);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] -= mean;
                s[0] += (S::kWhole ? c : c + j) < p.cols ? v[i][j] * v[i][j] : 0.0f;
            }
        }
        row_sums<S, 1>(s, red, 1);
        const float rstd = 1.0f / sqrtf(s[0] / n + p.eps);
        if (mine && l == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
        if (!mine) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t c = 8 * (l + S::kLanes * i);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * rstd, w[i][j], b[i][j]);
            if (p.out && c < p.cols)
                store_row8<IN, S::kWhole>(row_at<IN>(p.out, r, p.cols), c, p.cols, v[i], p.early);
            if constexpr (CODES) {
                const int64_t groups = (p.cols + kGroup - 1) / kGroup;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] = (S::kWhole ? c : c + j) < p.cols ? v[i][j] : 0.0f;
                // (16 lanes share a group, and all 16 are here)
                const Codes8 q = group_codes(p.fmt, v[i], p.rmargin);
                if (c < p.cols) store8(p.out8, r, c, p.cols, 0, q.lo, q.hi);
                if (l % 16 == 0 && c < p.cols) p.scale8[r * groups + c / kGroup] = q.step;
            }
        }
    }
}

// dx and the workgroup's share of dw and db: its rows' sums stay in
// registers, then the row places' are added up through LDS and written to
// part [workgroup][2][cols].
template <int IN, class S, bool SUMS>
__device__ __forceinline__ void bwd_rows(const NormBwdLaunch& p, int block, int blocks) {
    constexpr int V = S::kV, kCols = 8 * S::kLanes * V;
    __shared__ float red[2 * 2 * (S::kT / kWave)];
    __shared__ float fold[SUMS && S::kRows > 1 ? S::kRows : 1][2][SUMS && S::kRows > 1 ? kCols : 1];
    const int l = threadIdx.x % S::kLanes, place = threadIdx.x / S::kLanes;
    const int64_t step = (int64_t)blocks * S::kRows;
    const int64_t first = (int64_t)block * S::kRows;
    const float rn = 1.0f / (float)p.cols;
    float w[V][8], dw[V][8] = {}, db[V][8] = {};
#pragma unroll
    for (int i = 0; i < V; ++i)
        load_param<IN, S::kWhole>(p.weight, p.w_f32, 8 * (l + S::kLanes * i), p.cols, 1.0f, w[i]);
    RowRaw<IN, S> nx, ng;
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t r) __attribute__((always_inline)) {
        nx.load(row_at<IN>(p.x, r, p.ldx), l, p.cols);
        ng.load(row_at<IN>(p.g, r, p.ldg), l, p.cols);
        nmean = p.mean[r];
        nrstd = p.rstd[r];
    };
    // (no registers are left for a second row of 64 bytes a lane and operand)
    constexpr bool kAhead = IN != kInF32 || V < 4;
    if (kAhead && first + place < p.rows) fetch(first + place);
    int turn = 0;
    for (int64_t at = first; at < p.rows; at += step) {
        const int64_t r = at + place;
        const bool mine = r < p.rows;
        if (!kAhead && mine) fetch(r);
        RowRaw<IN, S> x = nx, g = ng;
        const float mean = nmean, rstd = nrstd;
        if (kAhead && r + step < p.rows) fetch(r + step);
        float s[2] = {0.0f, 0.0f};
        // h and v of column j of piece i
        const auto h = [&](int i, int j) { return (x.v[i][j] - mean) * rstd; };
        const auto v = [&](int i, int j) { return g.v[i][j] * w[i][j]; };
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[0] += v(i, j);
                s[1] = fmaf(v(i, j), h(i, j), s[1]);
            }
        }
        if (SUMS && mine) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dw[i][j] = fmaf(g.v[i][j], h(i, j), dw[i][j]);
                    db[i][j] += g.v[i][j];
                }
            }
        }
        // (long rows: h and v are computed twice, where kept ones would have to go
        // through memory)
        if constexpr (S::kTwice) {
            x.forget();
            g.forget();
        }
        if (!p.dx) continue;
        row_sums<S, 2>(s, red, turn);
        turn ^= 1;
        const float m0 = s[0] * rn, m1 = s[1] * rn;
        if (!mine) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t c = 8 * (l + S::kLanes * i);
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = rstd * (v(i, j) - fmaf(h(i, j), m1, m0));
            if (c < p.cols)
                store_row8<IN, S::kWhole>(row_at<IN>(p.dx, r, p.cols), c, p.cols, d, p.early);
        }
    }
    if constexpr (SUMS) {
        float* part = p.part + 2 * (int64_t)block * p.cols;
        if constexpr (S::kRows > 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = 8 * (l + S::kLanes * i) + j;
                    fold[place][0][c] = dw[i][j];
                    fold[place][1][c] = db[i][j];
                }
            }
            __syncthreads();
            for (int at = threadIdx.x; at < 2 * kCols; at += S::kT) {
                const int which = at / kCols, c = at % kCols;
                if (c >= p.cols) continue;
                float sum = fold[0][which][c];
#pragma unroll
                for (int k = 1; k < S::kRows; ++k) sum += fold[k][which][c];
                part[which * p.cols + c] = sum;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int64_t c = 8 * (l + S::kLanes * i);
                if (c >= p.cols) continue;
                store_row8<kInF32>(part, c, p.cols, dw[i]);
                store_row8<kInF32>(part + p.cols, c, p.cols, db[i]);
            }
        }
    }
}

template <int IN, class S, bool SUMS>
__global__ __launch_bounds__(S::kT) void norm_bwd_rows_kernel(NormBwdLaunch p) {
    bwd_rows<IN, S, SUMS>(p, blockIdx.x, gridDim.x);
}

template <int IN>
__device__ __forceinline__ void store_param(void* p, bool f32, int64_t c, float v) {
    if (f32 || IN == kInF32)
        static_cast<float*>(p)[c] = v;
    else if constexpr (IN == kInBf16)
        static_cast<uint16_t*>(p)[c] = f32_to_bf16(v);
    else
        static_cast<_Float16*>(p)[c] = (_Float16)v;
}

// dw and db of 32 columns from all rows: four lanes a row, eight rows under way
// at a time.
constexpr int kColCols = 32;

template <int IN, int T, bool WHOLE>
__device__ __forceinline__ void bwd_cols(const NormBwdLaunch& p, int block) {
    constexpr int kPlaces = T / 4, kAhead = 8, kWaves = T / kWave;
    __shared__ float red[kWaves][2][kColCols];
    const int place = threadIdx.x / 4, at = 8 * (threadIdx.x % 4);
    const int64_t c = (int64_t)block * kColCols + at;
    float dw[8] = {}, db[8] = {};
    if (c < p.cols) {
        for (int64_t r0 = place; r0 < p.rows; r0 += kAhead * kPlaces) {
            Raw8<IN> x[kAhead], g[kAhead];
            float mean[kAhead], rstd[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int64_t r = r0 + i * kPlaces;
                if (r >= p.rows) continue;
                x[i] = load_row8<IN, false, WHOLE>(row_at<IN>(p.x, r, p.ldx), c, p.cols);
                g[i] = load_row8<IN, false, WHOLE>(row_at<IN>(p.g, r, p.ldg), c, p.cols);
                mean[i] = p.mean[r];
                rstd[i] = p.rstd[r];
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (r0 + i * kPlaces >= p.rows) continue;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dw[j] = fmaf(g[i][j], (x[i][j] - mean[i]) * rstd[i], dw[j]);
                    db[j] += g[i][j];
                }
            }
        }
    }
    // the wave's sixteen places (lanes 4 apart), then the waves
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const auto add = [](float a, float b) { return a + b; };
        dw[j] += rotate16<8>(dw[j]);
        db[j] += rotate16<8>(db[j]);
        dw[j] = across_rows(dw[j] + rotate16<4>(dw[j]), add);
        db[j] = across_rows(db[j] + rotate16<4>(db[j]), add);
        if (threadIdx.x % kWave < 4) {
            red[threadIdx.x / kWave][0][at + j] = dw[j];
            red[threadIdx.x / kWave][1][at + j] = db[j];
        }
    }
    __syncthreads();
    if (threadIdx.x >= 2 * kColCols) return;
    const int which = threadIdx.x / kColCols, col = threadIdx.x % kColCols;
    const int64_t column = (int64_t)block * kColCols + col;
    void* out = which ? p.dbias : p.dweight;
    if (!out || column >= p.cols) return;
    float sum = red[0][which][col];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += red[w][which][col];
    store_param<IN>(out, p.w_f32, column, sum);
}

// Few rows: dw and db by workgroups of their own, which read x and g a second
// time (from the caches), so that nothing has to be added up in another launch
// (see both_at_once).
template <int IN, class S>
__global__ __launch_bounds__(S::kT) void norm_bwd_both_kernel(NormBwdLaunch p, int col_blocks) {
    if ((int)blockIdx.x < col_blocks)
        bwd_cols<IN, S::kT, S::kWhole>(p, blockIdx.x);
    else
        bwd_rows<IN, S, false>(p, blockIdx.x - col_blocks, gridDim.x - col_blocks);
}

// ---- rows of any length ---------------------------------------------------

// A workgroup per row, which it reads three times.
template <int IN>
__global__ __launch_bounds__(kT) void norm_fwd_kernel(NormFwdLaunch p) {
    __shared__ float red[kT / kWave];
    const int64_t r = workgroup_id();
    if (r >= p.rows) return;
    const void* x = row_at<IN>(p.x, r, p.ldx);
    const float n = (float)p.cols;
    float v[8], w[8], b[8], s = 0.0f;
    for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * kT) {
        load_row8<IN>(x, c, p.cols).values(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[j];
    }
    const float mean = block_sum<kT>(s, red) / n;
    s = 0.0f;
    for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * kT) {
        load_row8<IN>(x, c, p.cols).values(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s += c + j < p.cols ? (v[j] - mean) * (v[j] - mean) : 0.0f;
    }
    const float rstd = 1.0f / sqrtf(block_sum<kT>(s, red) / n + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[r] = mean;
        if (p.rstd) p.rstd[r] = rstd;
    }
    if (!p.out && !p.out8) return;
    const int64_t groups = (p.cols + kGroup - 1) / kGroup;
    // whole groups of 16 lanes take part in a group of columns
    for (int64_t c = 8 * threadIdx.x; c < groups * kGroup; c += 8 * kT) {
        load_row8<IN>(x, c, p.cols).values(v);
        load_param<IN>(p.weight, p.w_f32, c, p.cols, 1.0f, w);
        load_param<IN>(p.bias, p.w_f32, c, p.cols, 0.0f, b);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = c + j < p.cols ? fmaf((v[j] - mean) * rstd, w[j], b[j]) : 0.0f;
        if (p.out) store_row8<IN>(row_at<IN>(p.out, r, p.cols), c, p.cols, v);
        if (p.out8) {
            const Codes8 q = group_codes(p.fmt, v, p.rmargin);
            store8(p.out8, r, c, p.cols, 0, q.lo, q.hi);
            if (threadIdx.x % 16 == 0) p.scale8[r * groups + c / kGroup] = q.step;
        }
    }
}

// dx: a workgroup per row, which it reads twice.
template <int IN>
__global__ __launch_bounds__(kT) void norm_dx_kernel(NormBwdLaunch p) {
    __shared__ float red[kT / kWave];
    const int64_t r = workgroup_id();
    if (r >= p.rows) return;
    const void* x = row_at<IN>(p.x, r, p.ldx);
    const void* g = row_at<IN>(p.g, r, p.ldg);
    const float mean = p.mean[r], rstd = p.rstd[r], n = (float)p.cols;
    float xv[8], gv[8], w[8], s0 = 0.0f, s1 = 0.0f;
    for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * kT) {
        load_row8<IN>(x, c, p.cols).values(xv);
        load_row8<IN>(g, c, p.cols).values(gv);
        load_param<IN>(p.weight, p.w_f32, c, p.cols, 1.0f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c + j >= p.cols) continue;
            s0 += gv[j] * w[j];
            s1 = fmaf(gv[j] * w[j], (xv[j] - mean) * rstd, s1);
        }
    }
    const float m0 = block_sum<kT>(s0, red) / n;
    const float m1 = block_sum<kT>(s1, red) / n;
    for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * kT) {
        load_row8<IN>(x, c, p.cols).values(xv);
        load_row8<IN>(g, c, p.cols).values(gv);
        load_param<IN>(p.weight, p.w_f32, c, p.cols, 1.0f, w);
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            d[j] = rstd * (gv[j] * w[j] - m0 - (xv[j] - mean) * rstd * m1);
        store_row8<IN>(row_at<IN>(p.dx, r, p.cols), c, p.cols, d);
    }
}

// Partial sums over a chunk of rows, eight columns a lane: part [chunk][2][cols].
constexpr int64_t kChunks = 256;  // at most

constexpr int kDwT = 256, kDwCols = 8 * kDwT;

template <int IN>
__global__ __launch_bounds__(kDwT) void norm_dw_kernel(NormBwdLaunch p) {
    const int64_t c = (int64_t)blockIdx.x * kDwCols + 8 * threadIdx.x;
    const int64_t chunk = blockIdx.y;
    if (c >= p.cols) return;
    float dw[8] = {}, db[8] = {};
    const int64_t each = (p.rows + gridDim.y - 1) / gridDim.y;
    const int64_t last = (chunk + 1) * each < p.rows ? (chunk + 1) * each : p.rows;
    for (int64_t r = chunk * each; r < last; ++r) {
        const Raw8<IN> x = load_row8<IN>(row_at<IN>(p.x, r, p.ldx), c, p.cols);
        const Raw8<IN> g = load_row8<IN>(row_at<IN>(p.g, r, p.ldg), c, p.cols);
        const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[j] = fmaf(g[j], (x[j] - mean) * rstd, dw[j]);
            db[j] += g[j];
        }
    }
    float* part = p.part + 2 * chunk * p.cols;
    store_row8<kInF32>(part, c, p.cols, dw);
    store_row8<kInF32>(part + p.cols, c, p.cols, db);
}

// Adds up part [shares][2][cols].  A workgroup takes 64 columns of dw or db,
// four a lane; its 64 groups of 16 lanes take a share in 64 each, four of which
// are under way at once.
constexpr int kFinalT = 1024, kFinalGroups = kFinalT / 16, kFinalCols = 64;

template <int IN>
__global__ __launch_bounds__(kFinalT) void norm_sums_kernel(NormBwdLaunch p, int shares) {
    __shared__ float red[kFinalT / kWave][kFinalCols];
    const int lane = threadIdx.x % 16, group = threadIdx.x / 16, which = blockIdx.y;
    void* out = which ? p.dbias : p.dweight;
    if (!out) return;
    const int64_t c = (int64_t)blockIdx.x * kFinalCols + 4 * lane;
    const float* at = p.part + which * p.cols + c;
    float acc[4] = {};
    if (c + 4 <= p.cols) {
        for (int k = group; k < shares; k += 4 * kFinalGroups) {
            AnyVec4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = k + i * kFinalGroups;
                v[i] = s < shares ? *reinterpret_cast<const AnyVec4*>(at + 2 * (int64_t)s * p.cols)
                                  : AnyVec4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] += __uint_as_float(v[i][j]);
            }
        }
    } else {
        for (int k = group; k < shares; k += kFinalGroups) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < p.cols) acc[j] += at[2 * (int64_t)k * p.cols + j];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        acc[j] = across_rows(acc[j], [](float a, float b) { return a + b; });
        if (threadIdx.x % kWave < 16) red[threadIdx.x / kWave][4 * lane + j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x >= kFinalCols) return;
    const int64_t col = (int64_t)blockIdx.x * kFinalCols + threadIdx.x;
    if (col >= p.cols) return;
    float s = red[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kFinalT / kWave; ++w) s += red[w][threadIdx.x];
    store_param<IN>(out, p.w_f32, col, s);
}

// ---- launches ---------------------------------------------------------------

constexpr int64_t kRegisterCols = 16384;  // rows up to here are held in registers

// Row places that a launch needs, in workgroups.
template <class S>
int64_t workgroups_needed(int64_t rows) {
    return (rows + S::kRows - 1) / S::kRows;
}
constexpr int64_t kCus = 256;

// Forward: several workgroups for each CU at most, which go on to further rows.
template <class S>
int64_t fwd_workgroups(int64_t rows) {
    const int64_t need = workgroups_needed<S>(rows);
    return need < 4 * kCus ? need : 4 * kCus;
}

// Backward: one for each CU (each is a share of the parameters' gradients to be
// added up: with two 4096 x 8192 bf16 took 47 us, with one 41), and all go over
// the same number of rows: where those are few turns, fewer workgroups, whose shares
// are fewer to add up, take no longer than one on each CU with turns of uneven
// number.  So / uneven, us, bf16: 257 places (2056 x 1024) 129 workgroups 8.4 / 8.4;
// 288 (2300 x 1024) 8.6 / 9.3; 514 (4111 x 1000) 172 workgroups 11.0 / 11.7; 525 (4200 x
// 1024) 10.9 / 11.6; 775 (6200 x 1024) 13.3 / 13.5; 1030 x 8192 19.6 / 21.6; dx alone
// 257 places 4.8 / 4.3, 514 6.9 / 7.0.
template <class S>
int64_t bwd_workgroups(int64_t rows) {
    const int64_t need = workgroups_needed<S>(rows);
    const int64_t turns = (need + kCus - 1) / kCus;
    return (need + turns - 1) / turns;
}

// fn(Shape) for a row's length: the fewest lanes that hold it in registers with
// 8 or 16 columns each, 32 from 8192 on.  Forward / backward, us, bf16: 200000 x 64
// with 8 lanes 12.0 / 20.0, with 16 16.0 / 27.0; 65536 x 128 with 16 8.2 / 13.7, with 64
// 19.3 / 28.9; 100000 x 256 with 32 19.4 / 32.0, with 64 29.0 / 47.0; 16384 x 1024 with 64 15.7 / 23.2, with 256
// 21.7 / 32.5; 16384 x 2048 with 256 25.0 / 40.5, with 64 30.5 / 40.0; 4096 x 8192 with
// 512 25.9 / 41.4, with 256 33.0 / 46.0; 2048 x 16384 with 512 33 / 47, with 1024 (which
// have too few registers) 32 / 64.  Few rows of 4096 are shorter chains with 8 columns
// a lane.  512 / 256 lanes, forward: 16 rows 2.9 / 3.8, 2048 rows 7.8 / 9.9, 4096 rows
// 15.3 / 16.8, 16384 rows 53.7 / 49.5; backward: 16 rows 2.9 / 3.3, 256 rows 5.1 / 4.4,
// 1024 rows 13.4 / 13.3, 2048 rows 18.6 / 18.8, 4096 rows 25.4 / 24.6, 16384 rows 76.8 /
// 75.9.
constexpr int64_t kFewRows = 2048;
template <bool WHOLE, class Fn>
auto with_lanes(int64_t rows, int64_t cols, bool codes, Fn fn) {
    if (cols <= 64 && !codes) return fn(Shape<8, 1, WHOLE>{});
    if (cols <= 128) return fn(Shape<16, 1, WHOLE>{});
    if (cols <= 256) return fn(Shape<32, 1, WHOLE>{});
    if (cols <= 512) return fn(Shape<64, 1, WHOLE>{});
    if (cols <= 1024) return fn(Shape<64, 2, WHOLE>{});
    if (cols <= 2048) return fn(Shape<256, 1, WHOLE>{});
    if (cols <= 4096 && rows <= kFewRows) return fn(Shape<512, 1, WHOLE>{});
    if (cols <= 4096) return fn(Shape<256, 2, WHOLE>{});
    if (cols <= 8192) return fn(Shape<512, 2, WHOLE>{});
    return fn(Shape<512, 4, WHOLE>{});
}
// (whole groups of 8 need no guards: 4111 x 1000 fp16 6.6 / 11.3, with them 7.1 / 14.2)
template <class Fn>
auto with_shape(int64_t rows, int64_t cols, bool codes, Fn fn) {
    return cols % 8 == 0 ? with_lanes<true>(rows, cols, codes, fn)
                         : with_lanes<false>(rows, cols, codes, fn);
}

template <int IN>
hipError_t launch_fwd(const NormFwdLaunch& q, hipStream_t stream) {
    if (q.cols > kRegisterCols) {
        hipLaunchKernelGGL(norm_fwd_kernel<IN>, grid_of(q.rows), dim3(kT), 0, stream, q);
        return hipGetLastError();
    }
    return with_shape(q.rows, q.cols, q.out8 != nullptr, [&](auto shape) {
        using S = decltype(shape);
        const dim3 grid((unsigned)fwd_workgroups<S>(q.rows));
        if constexpr (S::kLanes >= 16) {  // (that hold whole groups of 128 between them)
            if (q.out8) {
                hipLaunchKernelGGL((norm_fwd_rows_kernel<IN, S, true>), grid, dim3(S::kT), 0,
                                   stream, q);
                return hipGetLastError();
            }
        }
        hipLaunchKernelGGL((norm_fwd_rows_kernel<IN, S, false>), grid, dim3(S::kT), 0, stream, q);
        return hipGetLastError();
    });
}

// Few enough rows for norm_bwd_both_kernel.  One launch / two, us in a graph, bf16:
// 64 x 1024 3.0 / 6.1, 256 x 4096 4.4 / 9.9, 1024 x 1024 6.5 / 7.2, 1024 x 4096 13.2 /
// 14.4, 300 x 8192 10.2 / 13.3; 1000 x 8192 23.8 / 20.7, 2048 x 1024 19.5 / 8.4 (rows of
// a power of two keep a few of the memory's channels busy, and ever longer).
constexpr int64_t kBothRows = 1024, kBothElements = 1 << 22;
bool both_at_once(int64_t rows, int64_t cols) {
    return cols <= kRegisterCols && rows <= kBothRows && rows * cols <= kBothElements;
}

// Shares of the parameters' gradients, to be added up in a second launch.
int64_t shares_of(int64_t rows, int64_t cols) {
    if (rows < 1 || both_at_once(rows, cols)) return 0;
    if (cols > kRegisterCols) return rows < kChunks ? rows : kChunks;
    return with_shape(rows, cols, false, [&](auto shape) {
        return bwd_workgroups<decltype(shape)>(rows);
    });
}

template <int IN>
hipError_t launch_bwd(const NormBwdLaunch& q, hipStream_t stream) {
    const bool sums = q.dweight || q.dbias;
    const int64_t shares = shares_of(q.rows, q.cols);
    if (sums && q.rows > 0 && both_at_once(q.rows, q.cols))
        return with_shape(q.rows, q.cols, false, [&](auto shape) {
            using S = decltype(shape);
            const int cols = (int)((q.cols + kColCols - 1) / kColCols);
            const int rows = q.dx ? (int)fwd_workgroups<S>(q.rows) : 0;
            hipLaunchKernelGGL((norm_bwd_both_kernel<IN, S>), dim3(cols + rows), dim3(S::kT), 0,
                               stream, q, cols);
            return hipGetLastError();
        });
    if (q.rows > 0 && q.cols <= kRegisterCols) {
        const hipError_t e = with_shape(q.rows, q.cols, false, [&](auto shape) {
            using S = decltype(shape);
            const dim3 grid((unsigned)bwd_workgroups<S>(q.rows));
            if (sums)
                hipLaunchKernelGGL((norm_bwd_rows_kernel<IN, S, true>), grid, dim3(S::kT), 0, stream, q);
            else
                hipLaunchKernelGGL((norm_bwd_rows_kernel<IN, S, false>), grid, dim3(S::kT), 0, stream, q);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    } else if (q.rows > 0) {
        if (q.dx) {
            hipLaunchKernelGGL(norm_dx_kernel<IN>, grid_of(q.rows), dim3(kT), 0, stream, q);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        if (sums) {
            const unsigned cols = (unsigned)((q.cols + kDwCols - 1) / kDwCols);
            hipLaunchKernelGGL(norm_dw_kernel<IN>, dim3(cols, (unsigned)shares), dim3(kDwT), 0,
                               stream, q);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    if (!sums) return hipSuccess;
    const unsigned blocks = (unsigned)((q.cols + kFinalCols - 1) / kFinalCols);
    hipLaunchKernelGGL(norm_sums_kernel<IN>, dim3(blocks, 2), dim3(kFinalT), 0, stream, q,
                       (int)shares);
    return hipGetLastError();
}

}  // namespace

size_t norm_bwd_partials(int64_t rows, int64_t cols) {
    return 2 * sizeof(float) * (size_t)shares_of(rows, cols) * (size_t)cols;
}

hipError_t launch_norm_fwd(const NormFwdLaunch& of, hipStream_t stream) {
    NormFwdLaunch q = of;
    q.early = written_early(q.rows * q.cols * size_of(q.type), q.cols * size_of(q.type));
    if (q.type == kInBf16) return launch_fwd<kInBf16>(q, stream);
    return q.type == kInF16 ? launch_fwd<kInF16>(q, stream) : launch_fwd<kInF32>(q, stream);
}

hipError_t launch_norm_bwd(const NormBwdLaunch& of, hipStream_t stream) {
    NormBwdLaunch q = of;
    q.early = written_early(q.rows * q.cols * size_of(q.type), q.cols * size_of(q.type));
    if (q.type == kInBf16) return launch_bwd<kInBf16>(q, stream);
    return q.type == kInF16 ? launch_bwd<kInF16>(q, stream) : launch_bwd<kInF32>(q, stream);
}

}  // namespace fp8lin
