// Block quantize: bf16 / fp16 / fp32 -> fp8 codes with one step for each
// group of 128 values, along rows (1 x 128), along columns (128 x 1) or for
// 128 x 128 tiles:
//     s = max(max |x| * fp32(1 / FMAX) * 2^-margin, 1e-12),   q = enc(x * fp32(1 / s)).
// (The step takes one multiplication where the per-tensor ring's fold takes a
// division, once per tensor: the two can differ in the last bit.)
//
// One workgroup of 256 lanes holds one 128 x 128 tile of x in registers
// (lane t: columns 8 (t % 16) .. +7 of rows t / 16 + 16 i), so x is read
// once whatever is asked: a row group's maximum is that of 16 neighbouring
// lanes, a column group's that of a lane's own 8 rows, of the 4 row lanes of
// its wave and, through LDS, of the 4 waves.  16 lanes read 256 bytes of a
// row (bf16) and write the 128 bytes of its codes: whole lines both ways.
// Memory bound: 3 bytes per element for one grouping of a 2-byte input, 4
// for both.

#include "block.hpp"
#include "common.hpp"

namespace fp8lin {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsPer = kThreads / 16;       // rows a pass of the workgroup covers
constexpr int kPasses = kGroup / kRowsPer;    // 8 rows per lane

struct BlockQuantParams {
    const void* x;
    int64_t rows, cols, ldx;
    int fmt;
    float rmargin;  // 2^-margin
    uint8_t* out_row;
    float* scale_row;
    uint8_t* out_col;
    float* scale_col;
    uint8_t* out_tile;
    float* scale_tile;
    int64_t col_groups;
    int vec_out;  // codes go out 8 at a time: cols % 8 == 0 and aligned outputs
};

template <int IN>
struct Elem;
template <>
struct Elem<kInBf16> {
    using T = uint16_t;
    __device__ static float f(T v) { return bf16_to_f32(v); }
};
template <>
struct Elem<kInF16> {
    using T = uint16_t;
    __device__ static float f(T v) { return (float)__builtin_bit_cast(_Float16, v); }
};
template <>
struct Elem<kInF32> {
    using T = float;
    __device__ static float f(T v) { return v; }
};

// The step of a group whose largest magnitude is amax.
__device__ __forceinline__ float step_of(float amax, float rfmax, float rmargin) {
    return fmaxf(amax * rfmax * rmargin, 1e-12f);
}

// Eight codes of one row: columns c .. c + 7, those past cols dropped.
__device__ __forceinline__ void store8(uint8_t* out, int64_t row, int64_t c, int64_t cols,
                                       int vec, uint32_t lo, uint32_t hi) {
    uint8_t* dst = out + row * cols + c;
    if (vec) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        return;
    }
    const uint64_t w = lo | (uint64_t)hi << 32;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j < cols) dst[j] = (uint8_t)(w >> (8 * j));
}

template <int IN, bool ROW, bool COL, bool TILE>
__global__ __launch_bounds__(kThreads) void quantize_block_kernel(BlockQuantParams p) {
    using E = Elem<IN>;
    using T = typename E::T;
    __shared__ float red[4][kGroup];
    const int tid = threadIdx.x;
    const int wave = tid / kWave;
    const int cl = 8 * (tid % 16);
    const int64_t cg = (int64_t)blockIdx.x % p.col_groups, rg = (int64_t)blockIdx.x / p.col_groups;
    const int64_t c = cg * kGroup + cl;
    const int64_t r0 = rg * kGroup + tid / 16;
    const float rfmax = p.fmt ? 1.0f / fmt_max<1>() : 1.0f / fmt_max<0>();
    const T* x = static_cast<const T*>(p.x);

    T raw[kPasses][8];
    const bool whole = c + 8 <= p.cols;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = r0 + kRowsPer * i;
        const T* src = x + r * p.ldx + c;
        if (r < p.rows && whole) {
            __builtin_memcpy(raw[i], src, sizeof raw[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) raw[i][j] = r < p.rows && c + j < p.cols ? src[j] : T(0);
        }
    }

    float rmax[kPasses];
    float cmax[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        rmax[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = fabsf(E::f(raw[i][j]));  // (fmaxf drops NaN)
            rmax[i] = fmaxf(rmax[i], v);
            if constexpr (COL) cmax[j] = fmaxf(cmax[j], v);
        }
    }

    // codes of pass i with the reciprocals m (one per column)
    auto encode = [&](int i, const float (&m)[8], uint32_t& lo, uint32_t& hi) {
        lo = cvt4_rt(p.fmt, E::f(raw[i][0]) * m[0], E::f(raw[i][1]) * m[1],
                     E::f(raw[i][2]) * m[2], E::f(raw[i][3]) * m[3]);
        hi = cvt4_rt(p.fmt, E::f(raw[i][4]) * m[4], E::f(raw[i][5]) * m[5],
                     E::f(raw[i][6]) * m[6], E::f(raw[i][7]) * m[7]);
    };

    if constexpr (ROW) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            float a = rmax[i];
#pragma unroll
            for (int off = 8; off >= 1; off >>= 1) a = fmaxf(a, __shfl_xor(a, off, kWave));
            const float s = step_of(a, rfmax, p.rmargin);
            const float inv = __fdiv_rn(1.0f, s);
            const float m[8] = {inv, inv, inv, inv, inv, inv, inv, inv};
            const int64_t r = r0 + kRowsPer * i;
            if (r < p.rows && c < p.cols) {
                uint32_t lo, hi;
                encode(i, m, lo, hi);
                store8(p.out_row, r, c, p.cols, p.vec_out, lo, hi);
                if (cl == 0) p.scale_row[r * p.col_groups + cg] = s;
            }
        }
    }
    if constexpr (COL) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a = cmax[j];
            a = fmaxf(a, __shfl_xor(a, 16, kWave));
            a = fmaxf(a, __shfl_xor(a, 32, kWave));
            if (tid % kWave < 16) red[wave][cl + j] = a;
        }
        __syncthreads();
        float m[8], s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = fmaxf(fmaxf(red[0][cl + j], red[1][cl + j]),
                                  fmaxf(red[2][cl + j], red[3][cl + j]));
            s[j] = step_of(a, rfmax, p.rmargin);
            m[j] = __fdiv_rn(1.0f, s[j]);
        }
        if (tid < 16) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < p.cols) p.scale_col[rg * p.cols + c + j] = s[j];
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int64_t r = r0 + kRowsPer * i;
            if (r < p.rows && c < p.cols) {
                uint32_t lo, hi;
                encode(i, m, lo, hi);
                store8(p.out_col, r, c, p.cols, p.vec_out, lo, hi);
            }
        }
    }
    if constexpr (TILE) {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) a = fmaxf(a, rmax[i]);
        a = wave_max(a);
        if (tid % kWave == 0) red[0][wave] = a;
        __syncthreads();
        a = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
        const float s = step_of(a, rfmax, p.rmargin);
        const float inv = __fdiv_rn(1.0f, s);
        const float m[8] = {inv, inv, inv, inv, inv, inv, inv, inv};
        if (tid == 0) p.scale_tile[rg * p.col_groups + cg] = s;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int64_t r = r0 + kRowsPer * i;
            if (r < p.rows && c < p.cols) {
                uint32_t lo, hi;
                encode(i, m, lo, hi);
                store8(p.out_tile, r, c, p.cols, p.vec_out, lo, hi);
            }
        }
    }
}

template <int IN>
hipError_t launch_in(const BlockQuantParams& p, int64_t grid, hipStream_t stream) {
    const dim3 g((unsigned)grid), b(kThreads);
    if (p.out_tile)
        hipLaunchKernelGGL((quantize_block_kernel<IN, false, false, true>), g, b, 0, stream, p);
    else if (p.out_row && p.out_col)
        hipLaunchKernelGGL((quantize_block_kernel<IN, true, true, false>), g, b, 0, stream, p);
    else if (p.out_row)
        hipLaunchKernelGGL((quantize_block_kernel<IN, true, false, false>), g, b, 0, stream, p);
    else
        hipLaunchKernelGGL((quantize_block_kernel<IN, false, true, false>), g, b, 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_block(const BlockQuantLaunch& q, hipStream_t stream) {
    BlockQuantParams p{};
    p.x = q.x;
    p.rows = q.rows;
    p.cols = q.cols;
    p.ldx = q.ldx;
    p.fmt = q.fmt;
    p.rmargin = q.rmargin;
    p.out_row = q.out_row;
    p.scale_row = q.scale_row;
    p.out_col = q.out_col;
    p.scale_col = q.scale_col;
    p.out_tile = q.out_tile;
    p.scale_tile = q.scale_tile;
    p.col_groups = groups_of(q.cols);
    const uintptr_t outs = reinterpret_cast<uintptr_t>(q.out_row) |
                           reinterpret_cast<uintptr_t>(q.out_col) |
                           reinterpret_cast<uintptr_t>(q.out_tile);
    p.vec_out = q.cols % 8 == 0 && (outs & 7) == 0;
    const int64_t grid = groups_of(q.rows) * p.col_groups;
    switch (q.in_type) {
        case kInBf16: return launch_in<kInBf16>(p, grid, stream);
        case kInF16: return launch_in<kInF16>(p, grid, stream);
        default: return launch_in<kInF32>(p, grid, stream);
    }
}

}  // namespace fp8lin
