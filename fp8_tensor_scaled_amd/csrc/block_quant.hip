// Block quantize: bf16 / fp16 / fp32 -> fp8 codes with one step for each
// group of 128 values, along rows (1 x 128), along columns (128 x 1) or for
// 128 x 128 tiles:
//     s = max(max |x| * fp32(1 / FMAX) * 2^-margin, 1e-12),   q = enc(x * fp32(1 / s)).
// (The step takes one multiplication by a rounded reciprocal where the per-tensor
// ring's fold takes a division, once per tensor: the two can differ in the last
// bit.  Of 4.2 M normal bf16 values, rows
// in groups, 5084 E4M3 codes lie on the other side of a tie than with an exact
// step, 2136 with a divided one; E5M2 4720 and 1168.)
//
// A workgroup of T lanes holds a band of 128 columns in registers (lane t:
// columns 8 (t % 16) .. +7 of rows t / 16 + (T / 16) i, i < P; 128 rows
// where columns or tiles are grouped), so x is read once whatever is asked.  A
// row group's maximum is that of 16 neighbouring lanes; a column group's that
// of a lane's own rows, of the 4 row lanes of its wave and, through LDS, of
// the waves.  16 lanes read 256 bytes of a row (2-byte inputs) and write the
// 128 bytes of its codes: whole lines both ways.  Each reciprocal (a
// correctly rounded division) is taken by one lane and handed to the others.
//
// Without a margin nothing has to be clamped before the conversion: |x| <=
// max |x| gives |x / s| <= FMAX (1 + 2^-22), which rounds to FMAX at most, and
// a larger step only lowers it.
//
// Memory bound when large (3 bytes per element for one grouping of a 2-byte
// input, 4 for both); a few tiles are bound by the chain of one tile (load,
// maxima, division, conversion), so there 1024 lanes share a tile instead of
// 256 (see launch_kinds).

#include "block.hpp"
#include "common.hpp"

namespace fp8lin {

namespace {

struct BlockQuantParams {
    const void* x;
    int64_t rows, cols, ldx;
    float rmargin;  // 2^-margin
    uint8_t* out_row;
    float* scale_row;
    uint8_t* out_col;
    float* scale_col;
    uint8_t* out_tile;
    float* scale_tile;
    float* sums;  // [groups_of(rows)][cols] column sums of x over each 128 rows
    int64_t col_groups;
    int64_t bands;  // workgroups of the launch (see grid_of)
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

// Four codes, without a clamp.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    int w;
    if constexpr (FMT) {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    }
    return (uint32_t)w;
}

// Eight codes of one row: columns c .. c + 7, those past cols dropped.
__device__ __forceinline__ void store8(uint8_t* out, int64_t row, int64_t c, int64_t cols,
                                       int vec, uint32_t lo, uint32_t hi) {
    uint8_t* dst = out + row * cols + c;
    if (vec) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        return;
    }
    if (c + 8 <= cols) {
        const uint2 w = make_uint2(lo, hi);
        __builtin_memcpy(dst, &w, 8);
        return;
    }
    const uint64_t w = lo | (uint64_t)hi << 32;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j < cols) dst[j] = (uint8_t)(w >> (8 * j));
}

// This lane's value from lane (its row of 16's first + N).
template <int N>
__device__ __forceinline__ float from_lane16(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + N, 0xf, 0xf,
                                                      false));  // row_newbcast:N
}
template <int N>
__device__ __forceinline__ float rotate16(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xf, 0xf,
                                                      false));  // row_ror:N
}
// op over the 16 lanes of a row, in every lane.
template <class Op>
__device__ __forceinline__ float all16(float v, Op op) {
    v = op(v, rotate16<8>(v));
    v = op(v, rotate16<4>(v));
    v = op(v, rotate16<2>(v));
    return op(v, rotate16<1>(v));
}
// op over lanes l, l ^ 16, l ^ 32, l ^ 48, in every lane.
template <class Op>
__device__ __forceinline__ float across_rows(float v, Op op) {
    const int a = __float_as_int(v);
    const auto s = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = op(__int_as_float(s[0]), __int_as_float(s[1]));
    const int b = __float_as_int(v);
    const auto t = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return op(__int_as_float(t[0]), __int_as_float(t[1]));
}

// 16 bytes at any element's address.
typedef uint32_t AnyVec4 __attribute__((ext_vector_type(4), aligned(2)));

template <int T>
struct QuantLds {
    float red[T / kWave][kGroup];
    float sum[T / kWave][kGroup];
    float inv[kGroup];
};

// The band of 128 columns of column group cg and the T / 16 * P rows from
// row r_first (with COL, TILE or SUM: the 128 rows of row group rg).
template <int IN, int FMT, bool ROW, bool COL, bool TILE, bool SUM, int T, int P>
__device__ __forceinline__ void quantize_band(const BlockQuantParams& p, int64_t cg, int64_t rg,
                                              QuantLds<T>& lds) {
    using E = Elem<IN>;
    using V = typename E::T;
    constexpr int kRowsPer = T / 16, NW = T / kWave;
    static_assert(!(COL || TILE || SUM) || kRowsPer * P == kGroup, "a whole group of rows");
    constexpr float rfmax = 1.0f / fmt_max<FMT>();
    auto max2 = [](float a, float b) { return fmaxf(a, b); };
    auto add2 = [](float a, float b) { return a + b; };
    const int tid = threadIdx.x;
    const int wave = tid / kWave;
    const int cl = 8 * (tid % 16);
    const int64_t c = cg * kGroup + cl;
    const int64_t r0 = rg * (kRowsPer * P) + tid / 16;
    const V* x = static_cast<const V*>(p.x);

    V raw[P][8];
    constexpr int kLoads = (int)sizeof(V) * 8 / 16;  // 16-byte loads of a row
    AnyVec4 v[P][kLoads];
    const bool whole = c + 8 <= p.cols;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int64_t r = r0 + kRowsPer * i;
        const V* src = x + r * p.ldx + c;
        if (r < p.rows && whole) {
            // read once: past the caches (8192 x 8192 bf16 tiles 35 us, 51 without;
            // fp32 58 either way)
#pragma unroll
            for (int z = 0; z < kLoads; ++z)
                v[i][z] = __builtin_nontemporal_load(reinterpret_cast<const AnyVec4*>(src) + z);
            __builtin_memcpy(raw[i], v[i], sizeof raw[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) raw[i][j] = r < p.rows && c + j < p.cols ? src[j] : V(0);
        }
    }

    float rmax[P], cmax[8], csum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[j] = csum[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        rmax[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = E::f(raw[i][j]);
            if constexpr (ROW || TILE) rmax[i] = fmaxf(rmax[i], fabsf(v));  // (drops NaN)
            if constexpr (COL) cmax[j] = fmaxf(cmax[j], fabsf(v));
            if constexpr (SUM) csum[j] += v;
        }
    }
    // codes of row i with the reciprocals m (one per column)
    auto write = [&](uint8_t* out, int i, const float (&m)[8]) __attribute__((always_inline)) {
        const int64_t r = r0 + kRowsPer * i;
        if (r >= p.rows || c >= p.cols) return;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = E::f(raw[i][j]) * m[j];
        if (p.rmargin != 1.0f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = sat<FMT>(v[j]);
        }
        store8(out, r, c, p.cols, p.vec_out, encode4<FMT>(v[0], v[1], v[2], v[3]),
               encode4<FMT>(v[4], v[5], v[6], v[7]));
    };

    if constexpr (COL || SUM) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (COL) cmax[j] = across_rows(cmax[j], max2);
            if constexpr (SUM) csum[j] = across_rows(csum[j], add2);
        }
        if (tid % kWave < 16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (COL) lds.red[wave][cl + j] = cmax[j];
                if constexpr (SUM) lds.sum[wave][cl + j] = csum[j];
            }
        }
        __syncthreads();
        if (tid < kGroup) {
            const int64_t col = cg * kGroup + tid;
            if constexpr (COL) {
                float a = lds.red[0][tid];
#pragma unroll
                for (int w = 1; w < NW; ++w) a = fmaxf(a, lds.red[w][tid]);
                const float s = step_of(a, rfmax, p.rmargin);
                lds.inv[tid] = __fdiv_rn(1.0f, s);
                if (col < p.cols) p.scale_col[rg * p.cols + col] = s;
            }
            if constexpr (SUM) {
                float a = lds.sum[0][tid];
#pragma unroll
                for (int w = 1; w < NW; ++w) a += lds.sum[w][tid];
                if (col < p.cols) p.sums[rg * p.cols + col] = a;
            }
        }
        if constexpr (COL) __syncthreads();
    }
    if constexpr (ROW) {
        float inv[P];
        // lane i of a row of 16 divides for row i, all of them for few rows
        float mine = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            rmax[i] = all16(rmax[i], max2);
            mine = tid % 16 == i || P == 1 ? rmax[i] : mine;
        }
        const float s = step_of(mine, rfmax, p.rmargin);
        const float r1 = __fdiv_rn(1.0f, s);
        inv[0] = from_lane16<0>(r1);
        if constexpr (P > 1) inv[1] = from_lane16<1>(r1);
        if constexpr (P > 2) {
            static_assert(P <= 2 || P == 8, "rows per lane");
            inv[2] = from_lane16<2>(r1);
            inv[3] = from_lane16<3>(r1);
            inv[4] = from_lane16<4>(r1);
            inv[5] = from_lane16<5>(r1);
            inv[6] = from_lane16<6>(r1);
            inv[7] = from_lane16<7>(r1);
        }
        if (tid % 16 < P) {
            const int64_t r = r0 + kRowsPer * (tid % 16);
            if (r < p.rows) p.scale_row[r * p.col_groups + cg] = s;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float m[8] = {inv[i], inv[i], inv[i], inv[i], inv[i], inv[i], inv[i], inv[i]};
            write(p.out_row, i, m);
        }
    }
    if constexpr (COL) {
        float m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = lds.inv[cl + j];
#pragma unroll
        for (int i = 0; i < P; ++i) write(p.out_col, i, m);
    }
    if constexpr (TILE) {
        float a = rmax[0];
#pragma unroll
        for (int i = 1; i < P; ++i) a = fmaxf(a, rmax[i]);
        a = across_rows(all16(a, max2), max2);
        if (tid % kWave == 0) lds.red[0][wave] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w) a = fmaxf(a, lds.red[0][w]);
        const float s = step_of(a, rfmax, p.rmargin);
        const float r1 = __fdiv_rn(1.0f, s);
        const float m[8] = {r1, r1, r1, r1, r1, r1, r1, r1};
        if (tid == 0) p.scale_tile[rg * p.col_groups + cg] = s;
#pragma unroll
        for (int i = 0; i < P; ++i) write(p.out_tile, i, m);
    }
}

// Workgroups in a grid: past kGridX of them by rows of kGridX.  (A grid dimension
// counts lanes in 32 bits: 2^24 workgroups of 256 lanes would be none.)
constexpr int64_t kGridX = 1 << 21;
dim3 grid_of(int64_t workgroups) {
    if (workgroups <= kGridX) return dim3((unsigned)workgroups);
    return dim3((unsigned)kGridX, (unsigned)((workgroups + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t workgroup_id() {
    return (int64_t)blockIdx.y * kGridX + blockIdx.x;
}

template <int IN, int FMT, bool ROW, bool COL, bool TILE, bool SUM, int T, int P>
__global__ __launch_bounds__(T) void quantize_block_kernel(BlockQuantParams p) {
    __shared__ QuantLds<T> lds;
    const int64_t id = workgroup_id();
    if (id >= p.bands) return;
    quantize_band<IN, FMT, ROW, COL, TILE, SUM, T, P>(p, id % p.col_groups, id / p.col_groups, lds);
}

// The layer's forward: x by rows (and columns, WITH_COL) and w by tiles in
// one launch, x's bands first.
template <int FMT, bool WITH_COL, int T, int P>
__global__ __launch_bounds__(T) void quantize_block_two_kernel(BlockQuantParams px,
                                                              BlockQuantParams pw) {
    __shared__ QuantLds<T> lds;
    const int64_t id = workgroup_id(), of_w = id - px.bands;
    if (of_w < 0)
        quantize_band<kInBf16, FMT, true, WITH_COL, false, false, T, P>(
            px, id % px.col_groups, id / px.col_groups, lds);
    else if (of_w < pw.bands)
        quantize_band<kInBf16, FMT, false, false, true, false, T, P>(
            pw, of_w % pw.col_groups, of_w / pw.col_groups, lds);
}

BlockQuantParams params_of(const BlockQuantLaunch& q) {
    BlockQuantParams p{};
    p.x = q.x;
    p.rows = q.rows;
    p.cols = q.cols;
    p.ldx = q.ldx;
    p.rmargin = q.rmargin;
    p.out_row = q.out_row;
    p.scale_row = q.scale_row;
    p.out_col = q.out_col;
    p.scale_col = q.scale_col;
    p.out_tile = q.out_tile;
    p.scale_tile = q.scale_tile;
    p.sums = q.sums;
    p.col_groups = groups_of(q.cols);
    p.bands = groups_of(q.rows) * p.col_groups;
    const uintptr_t outs = reinterpret_cast<uintptr_t>(q.out_row) |
                           reinterpret_cast<uintptr_t>(q.out_col) |
                           reinterpret_cast<uintptr_t>(q.out_tile);
    p.vec_out = q.cols % 8 == 0 && (outs & 7) == 0;
    return p;
}

// Below this many tiles a tile has 1024 lanes, from it on 256; rows alone, which
// need no 128-row span, have 256 lanes per 16 rows of a tile below it.  bf16, us,
// the first way / 256 lanes a tile: both ways 256 x 256 (4 tiles) 4.2 / 4.8, 2048 x
// 2048 (256) 6.9 / 7.7, 2048 x 4096 (512) 10.2 / 10.7, 4096 x 4096 (1024) 17.8 / 14.3;
// tiles 3.0 / 3.3, 4.5 / 4.9, 6.8 / 7.2, 11.2 / 10.7, 8192 x 8192 37.2 / 35.1; rows
// 2.4 / 3.4, 4.9 / 5.3, 8.3 / 8.0, 13.1 / 11.7.
constexpr int64_t kManyTiles = 512;

template <int IN, int FMT, bool ROW, bool COL, bool TILE, bool SUM>
hipError_t launch_kinds(BlockQuantParams p, hipStream_t stream) {
    const int64_t tiles = p.bands;
    if constexpr (ROW && !COL && !SUM) {
        if (tiles < kManyTiles) {
            p.bands = (p.rows + 15) / 16 * p.col_groups;
            hipLaunchKernelGGL((quantize_block_kernel<IN, FMT, true, false, false, false, 256, 1>),
                               grid_of(p.bands), dim3(256), 0, stream, p);
        } else {
            hipLaunchKernelGGL((quantize_block_kernel<IN, FMT, true, false, false, false, 256, 8>),
                               grid_of(tiles), dim3(256), 0, stream, p);
        }
    } else if (tiles < kManyTiles) {
        hipLaunchKernelGGL((quantize_block_kernel<IN, FMT, ROW, COL, TILE, SUM, 1024, 2>),
                           grid_of(tiles), dim3(1024), 0, stream, p);
    } else {
        hipLaunchKernelGGL((quantize_block_kernel<IN, FMT, ROW, COL, TILE, SUM, 256, 8>),
                           grid_of(tiles), dim3(256), 0, stream, p);
    }
    return hipGetLastError();
}

template <int IN, int FMT>
hipError_t launch_in(const BlockQuantParams& p, hipStream_t stream) {
    if (p.out_tile) return launch_kinds<IN, FMT, false, false, true, false>(p, stream);
    if constexpr (IN == kInBf16) {
        if (p.sums) return launch_kinds<IN, FMT, true, true, false, true>(p, stream);
    }
    if (p.out_row && p.out_col) return launch_kinds<IN, FMT, true, true, false, false>(p, stream);
    if (p.out_row) return launch_kinds<IN, FMT, true, false, false, false>(p, stream);
    return launch_kinds<IN, FMT, false, true, false, false>(p, stream);
}

template <int FMT, bool WITH_COL>
hipError_t launch_two(const BlockQuantParams& px, const BlockQuantParams& pw, hipStream_t stream) {
    const int64_t tiles = px.bands + pw.bands;
    if (tiles < kManyTiles)
        hipLaunchKernelGGL((quantize_block_two_kernel<FMT, WITH_COL, 1024, 2>), grid_of(tiles),
                           dim3(1024), 0, stream, px, pw);
    else
        hipLaunchKernelGGL((quantize_block_two_kernel<FMT, WITH_COL, 256, 8>), grid_of(tiles),
                           dim3(256), 0, stream, px, pw);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_block(const BlockQuantLaunch& q, hipStream_t stream) {
    const BlockQuantParams p = params_of(q);
    switch (q.in_type) {
        case kInBf16: return q.fmt ? launch_in<kInBf16, 1>(p, stream) : launch_in<kInBf16, 0>(p, stream);
        case kInF16: return q.fmt ? launch_in<kInF16, 1>(p, stream) : launch_in<kInF16, 0>(p, stream);
        default: return q.fmt ? launch_in<kInF32, 1>(p, stream) : launch_in<kInF32, 0>(p, stream);
    }
}

hipError_t launch_quantize_block_two(const BlockQuantLaunch& x, const BlockQuantLaunch& w,
                                     hipStream_t stream) {
    const BlockQuantParams px = params_of(x), pw = params_of(w);
    if (x.fmt) return x.out_col ? launch_two<1, true>(px, pw, stream) : launch_two<1, false>(px, pw, stream);
    return x.out_col ? launch_two<0, true>(px, pw, stream) : launch_two<0, false>(px, pw, stream);
}

}  // namespace fp8lin
