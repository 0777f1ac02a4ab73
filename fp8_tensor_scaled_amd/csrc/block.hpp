// Block-scaled operators: launch interfaces (quantize with a step for each
// group of 128 values, the matrix product of such operands, and the
// mixture-of-experts layer on tile-scaled weights).
#pragma once

#include "internal.hpp"

namespace fp8lin {

constexpr int kGroup = 128;  // values per step along a row or a column
inline int64_t groups_of(int64_t n) { return (n + kGroup - 1) / kGroup; }

struct BlockQuantLaunch {
    const void* x = nullptr;  // [rows][cols], row stride ldx (elements)
    int in_type = kInBf16;
    int64_t rows = 0, cols = 0, ldx = 0;
    int fmt = 0;
    float rmargin = 1.0f;  // 2^-margin
    // Any one of row / col / tile, or row and col together.
    uint8_t* out_row = nullptr;   // [rows][cols]
    float* scale_row = nullptr;   // [rows][groups_of(cols)]
    uint8_t* out_col = nullptr;   // [rows][cols]
    float* scale_col = nullptr;   // [groups_of(rows)][cols]
    uint8_t* out_tile = nullptr;  // [rows][cols]
    float* scale_tile = nullptr;  // [groups_of(rows)][groups_of(cols)]
    // With row and col of a bf16 input: receives the sums of each 128 rows of
    // each column, [groups_of(rows)][cols] (the bias gradient's partials).
    float* sums = nullptr;
};
hipError_t launch_quantize_block(const BlockQuantLaunch& q, hipStream_t stream);
// Two bf16 quantizes of one format in one launch: x by rows (and columns),
// w by tiles; the results are those of two launches.
hipError_t launch_quantize_block_two(const BlockQuantLaunch& x, const BlockQuantLaunch& w,
                                     hipStream_t stream);

// Where the step of output row i (or column j) and k group kb lies:
// scale[(i >> shift) * si + kb * sk].
struct BlockScale {
    const float* s = nullptr;
    int shift = 0;  // 0: one step per row / column, 7: one per 128 of them
    int64_t si = 0, sk = 0;
};

struct BlockGemmLaunch {
    const uint8_t* a = nullptr;
    const uint8_t* b = nullptr;
    int fmt_a = 0, fmt_b = 0;
    int trans_a = 0, trans_b = 0;
    int64_t m = 0, n = 0, k = 0, lda = 0, ldb = 0;
    BlockScale sa, sb;
    const uint16_t* bias = nullptr;
    uint16_t* out = nullptr;
    // For a split along k: a counter per tile (zero between calls) and
    // block_gemm_partials bytes for the shares' sums; null: no split.
    uint32_t* counters = nullptr;
    float* part = nullptr;
};
constexpr size_t kSplitCounterBytes = 4 * 256;  // at most so many tiles are split
size_t block_gemm_partials(int64_t m, int64_t n, int64_t k);  // 0: no split
hipError_t launch_block_gemm(const BlockGemmLaunch& g, hipStream_t stream);
// A linear backward's dX (NN) and dW (TN) and, with cf.db, the last pass of
// its bias gradient: one launch where the tiled kernels take both.
hipError_t launch_block_gemm_pair(const BlockGemmLaunch& dx, const BlockGemmLaunch& dw,
                                  const ColsumFinalJob& cf, hipStream_t stream);
// (what that launch is, where it is one)
hipError_t launch_block_pair(const BlockGemmLaunch& dx, const BlockGemmLaunch& dw,
                             const ColsumFinalJob& cf, hipStream_t stream);

struct MoeLaunch {
    const uint16_t* x = nullptr;       // bf16 [tokens][dim]
    const uint16_t* router = nullptr;  // bf16 [experts][dim]
    const uint8_t* w13 = nullptr;      // codes [experts][2 * hidden][dim], gate rows first
    const float* s13 = nullptr;        // [experts][groups_of(2 * hidden)][groups_of(dim)]
    const uint8_t* w2 = nullptr;       // codes [experts][dim][hidden]
    const float* s2 = nullptr;         // [experts][groups_of(dim)][groups_of(hidden)]
    int tokens = 0, experts = 0, top_k = 0, dim = 0, hidden = 0, fmt = 0;
    bool renorm = false;
    void* ws = nullptr;
    uint16_t* out = nullptr;    // bf16 [tokens][dim]
    int32_t* ids = nullptr;     // [tokens][top_k], nullable
    float* weights = nullptr;   // [tokens][top_k], nullable
};
size_t moe_workspace(int64_t tokens, int64_t experts, int64_t top_k, int64_t dim, int64_t hidden);
hipError_t launch_moe(const MoeLaunch& g, hipStream_t stream);

}  // namespace fp8lin
