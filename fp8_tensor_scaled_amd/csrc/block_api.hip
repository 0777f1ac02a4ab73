// C entry points of the block-scaled operators: argument validation and the
// hand-over to the launches.  Declarations and contracts: fp8lin.h.

#include <hip/hip_runtime.h>

#include <math.h>

#include "../../include/fp8lin.h"
#include "api_util.hpp"
#include "block.hpp"

using fp8lin::check_device;
using fp8lin::clear_error;
using fp8lin::fail;
using fp8lin::fmt_ok;
using fp8lin::groups_of;
using fp8lin::hip_fail;

extern "C" {

fp8_status_t fp8_quantize_block(const void* x, fp8_in_t in_type, int64_t rows, int64_t cols,
                                int64_t ldx, fp8_fmt_t fmt, int32_t margin, uint8_t* out_row,
                                float* scale_row, uint8_t* out_col, float* scale_col,
                                uint8_t* out_tile, float* scale_tile, hipStream_t stream) {
    clear_error();
    const char* who = "fp8_quantize_block";
    if (!fmt_ok(fmt)) return fail(FP8_EINVAL, "%s: unsupported fp8 format %d", who, fmt);
    if (in_type != FP8_IN_BF16 && in_type != FP8_IN_F16 && in_type != FP8_IN_F32)
        return fail(FP8_EINVAL, "%s: unsupported input type %d", who, (int)in_type);
    if (rows < 0 || cols < 0)
        return fail(FP8_EINVAL, "%s: rows, cols must be >= 0 (got %lld, %lld)", who,
                    (long long)rows, (long long)cols);
    if (ldx < cols)
        return fail(FP8_EINVAL, "%s: ldx %lld < cols %lld", who, (long long)ldx,
                    (long long)cols);
    if ((double)rows * (double)ldx >= 9.0e15)
        return fail(FP8_EINVAL, "%s: too many elements", who);
    if (margin < 0 || margin > 64)
        return fail(FP8_EINVAL, "%s: margin %d outside [0, 64]", who, margin);
    if (rows == 0 || cols == 0) return FP8_OK;  // (empty tensors may have no address)
    if ((out_row == nullptr) != (scale_row == nullptr) ||
        (out_col == nullptr) != (scale_col == nullptr) ||
        (out_tile == nullptr) != (scale_tile == nullptr))
        return fail(FP8_EINVAL, "%s: codes and steps of a grouping go together", who);
    if (!out_row && !out_col && !out_tile) return fail(FP8_EINVAL, "%s: no output given", who);
    if (out_tile && (out_row || out_col))
        return fail(FP8_EINVAL, "%s: tiles go alone (rows and columns may go together)", who);
    if (!x) return fail(FP8_EINVAL, "%s: x is NULL", who);
    if ((uintptr_t)x % (in_type == FP8_IN_F32 ? 4 : 2))
        return fail(FP8_EINVAL, "%s: x is not aligned to its elements", who);
    if (((uintptr_t)scale_row | (uintptr_t)scale_col | (uintptr_t)scale_tile) & 3)
        return fail(FP8_EINVAL, "%s: a scale is not aligned to its elements", who);
    if ((double)groups_of(rows) * (double)groups_of(cols) >= 2147483647.0)
        return fail(FP8_EINVAL, "%s: too many blocks", who);
    if (out_row && out_col) {
        const uintptr_t a = (uintptr_t)out_row, b = (uintptr_t)out_col;
        const uintptr_t n = (uintptr_t)(rows * cols);
        if (a < b + n && b < a + n)
            return fail(FP8_EINVAL, "%s: out_row and out_col overlap", who);
    }
    fp8_status_t st = check_device();
    if (st) return st;
    fp8lin::BlockQuantLaunch q;
    q.x = x;
    q.in_type = in_type;
    q.rows = rows;
    q.cols = cols;
    q.ldx = ldx;
    q.fmt = fmt;
    q.rmargin = ldexpf(1.0f, -margin);
    q.out_row = out_row;
    q.scale_row = scale_row;
    q.out_col = out_col;
    q.scale_col = scale_col;
    q.out_tile = out_tile;
    q.scale_tile = scale_tile;
    hipError_t e = fp8lin::launch_quantize_block(q, stream);
    return e == hipSuccess ? FP8_OK : hip_fail(e, "block quantize launch");
}

size_t fp8_mm_block_workspace(int64_t m, int64_t n, int64_t k) {
    if (m < 1 || n < 1 || k < 1) return 0;
    const size_t part = fp8lin::block_gemm_partials(m, n, k);
    return part ? fp8lin::kSplitCounterBytes + part : 0;
}

}  // extern "C"

namespace {

// Where a step lies (BlockScale) for an operand whose rows (of A, columns of
// B) number `lines`, stored with the lines contiguous along k or across it.
fp8lin::BlockScale scale_of(const float* s, fp8_group_t group, bool k_major, int64_t lines,
                            int64_t k) {
    fp8lin::BlockScale r;
    r.s = s;
    r.shift = group == FP8_GROUP_TILE ? 7 : 0;
    const int64_t along = group == FP8_GROUP_TILE ? groups_of(lines) : lines;
    r.si = k_major ? groups_of(k) : 1;
    r.sk = k_major ? 1 : along;
    return r;
}

}  // namespace

extern "C" {

fp8_status_t fp8_mm_block(const uint8_t* a, const uint8_t* b, fp8_fmt_t fmt_a, fp8_fmt_t fmt_b,
                          int32_t trans_a, int32_t trans_b, int64_t m, int64_t n, int64_t k,
                          int64_t lda, int64_t ldb, const float* scale_a, fp8_group_t group_a,
                          const float* scale_b, fp8_group_t group_b, const uint16_t* bias,
                          uint16_t* out, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
    clear_error();
    const char* who = "fp8_mm_block";
    if (!fmt_ok(fmt_a) || !fmt_ok(fmt_b))
        return fail(FP8_EINVAL, "%s: unsupported fp8 format %d, %d", who, fmt_a, fmt_b);
    if (!a || !b || !out || !scale_a || !scale_b)
        return fail(FP8_EINVAL, "%s: NULL operand, output or scale", who);
    if ((trans_a != 0 && trans_a != 1) || (trans_b != 0 && trans_b != 1))
        return fail(FP8_EINVAL, "%s: trans flags must be 0 or 1", who);
    if ((group_a != FP8_GROUP_LINE && group_a != FP8_GROUP_TILE) ||
        (group_b != FP8_GROUP_LINE && group_b != FP8_GROUP_TILE))
        return fail(FP8_EINVAL, "%s: unsupported grouping %d, %d", who, (int)group_a,
                    (int)group_b);
    if (m < 1 || n < 1 || k < 1)
        return fail(FP8_EINVAL, "%s: m, n, k must be >= 1 (got %lld, %lld, %lld)", who,
                    (long long)m, (long long)n, (long long)k);
    const int64_t a_cols = trans_a ? m : k, b_cols = trans_b ? k : n;
    if (lda < a_cols)
        return fail(FP8_EINVAL, "%s: lda %lld < %lld", who, (long long)lda, (long long)a_cols);
    if (ldb < b_cols)
        return fail(FP8_EINVAL, "%s: ldb %lld < %lld", who, (long long)ldb, (long long)b_cols);
    if (lda >= (1 << 24) || ldb >= (1 << 24))
        return fail(FP8_EINVAL, "%s: lda, ldb must be below 2^24", who);
    if ((double)m * (double)n >= 1099511627776.0 ||
        (double)(trans_a ? k : m) * (double)lda >= 9.0e15 ||
        (double)(trans_b ? n : k) * (double)ldb >= 9.0e15)
        return fail(FP8_EINVAL, "%s: operand or output too large", who);
    if (((uintptr_t)out | (uintptr_t)bias) & 1)
        return fail(FP8_EINVAL, "%s: out or bias is not aligned to its elements", who);
    if (((uintptr_t)scale_a | (uintptr_t)scale_b) & 3)
        return fail(FP8_EINVAL, "%s: a scale is not aligned to its elements", who);
    const size_t need = fp8_mm_block_workspace(m, n, k);
    if (workspace) {
        if (workspace_bytes < need)
            return fail(FP8_EINVAL, "%s: workspace %zu < %zu bytes", who, workspace_bytes, need);
        if ((uintptr_t)workspace & 255)
            return fail(FP8_EINVAL, "%s: workspace not 256-byte aligned", who);
    }
    fp8_status_t st = check_device();
    if (st) return st;
    fp8lin::BlockGemmLaunch g;
    g.a = a;
    g.b = b;
    g.fmt_a = fmt_a;
    g.fmt_b = fmt_b;
    g.trans_a = trans_a;
    g.trans_b = trans_b;
    g.m = m;
    g.n = n;
    g.k = k;
    g.lda = lda;
    g.ldb = ldb;
    g.sa = scale_of(scale_a, group_a, trans_a == 0, m, k);
    g.sb = scale_of(scale_b, group_b, trans_b != 0, n, k);
    g.bias = bias;
    g.out = out;
    if (need && workspace) {
        g.counters = static_cast<uint32_t*>(workspace);
        g.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                          fp8lin::kSplitCounterBytes);
    }
    hipError_t e = fp8lin::launch_block_gemm(g, stream);
    return e == hipSuccess ? FP8_OK : hip_fail(e, "block gemm launch");
}

}  // extern "C"

namespace {

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// What the forward leaves for the backward: x's codes and steps by columns
// (for dW), w's by tiles (for dX, when they are made here).
struct SavedLayout {
    size_t x8, sx, w8, sw, total;
};
SavedLayout saved_layout(int64_t M, int64_t N, int64_t K, bool want_dx, bool want_dw) {
    SavedLayout l{};
    size_t at = 0;
    if (want_dw) {
        l.x8 = at;
        at = up256(at + (size_t)M * K);
        l.sx = at;
        at = up256(at + 4 * (size_t)groups_of(M) * K);
    }
    if (want_dx) {
        l.w8 = at;
        at = up256(at + (size_t)N * K);
        l.sw = at;
        at = up256(at + 4 * (size_t)groups_of(N) * groups_of(K));
    }
    l.total = at;
    return l;
}

// Workspaces begin with the per-tensor layer's control block, which these
// calls leave alone (it stays zero), so that both can share one.
constexpr size_t kControl = 6656;
struct FwdWs {
    size_t x8, sx, w8, sw, total;
};
FwdWs fwd_ws(int64_t M, int64_t N, int64_t K) {
    FwdWs l;
    l.x8 = kControl;
    l.sx = up256(l.x8 + (size_t)M * K);
    l.w8 = up256(l.sx + 4 * (size_t)M * groups_of(K));
    l.sw = up256(l.w8 + (size_t)N * K);
    l.total = up256(l.sw + 4 * (size_t)groups_of(N) * groups_of(K));
    return l;
}
struct BwdWs {
    size_t g8, sg, g8c, sgc, sums, total;
};
BwdWs bwd_ws(int64_t M, int64_t N) {
    BwdWs l;
    l.g8 = kControl;
    l.sg = up256(l.g8 + (size_t)M * N);
    l.g8c = up256(l.sg + 4 * (size_t)M * groups_of(N));
    l.sgc = up256(l.g8c + (size_t)M * N);
    l.sums = up256(l.sgc + 4 * (size_t)groups_of(M) * N);
    const size_t sums = 4 * (size_t)groups_of(M) * N, colsum = fp8lin::colsum_workspace(M, N);
    l.total = up256(l.sums + (sums > colsum ? sums : colsum));
    return l;
}

fp8_status_t check_layer(const char* who, int64_t M, int64_t N, int64_t K, int32_t margin) {
    if (M < 1 || N < 1 || K < 1)
        return fail(FP8_EINVAL, "%s: M, N, K must be >= 1 (got %lld, %lld, %lld)", who,
                    (long long)M, (long long)N, (long long)K);
    // N and K are row strides of the products' operands (see fp8_mm_block)
    if (N >= (1 << 24) || K >= (1 << 24))
        return fail(FP8_EINVAL, "%s: N and K must be below 2^24 (got %lld, %lld)", who,
                    (long long)N, (long long)K);
    const double lim = 1099511627776.0;
    if ((double)M * N >= lim || (double)M * K >= lim || (double)N * K >= lim)
        return fail(FP8_EINVAL, "%s: a matrix is too large", who);
    const double blocks = 2147483647.0 / 2;
    if ((double)groups_of(M) * groups_of(N) >= blocks ||
        (double)groups_of(M) * groups_of(K) >= blocks ||
        (double)groups_of(N) * groups_of(K) >= blocks)
        return fail(FP8_EINVAL, "%s: too many blocks", who);
    if (margin < 0 || margin > 64)
        return fail(FP8_EINVAL, "%s: margin %d outside [0, 64]", who, margin);
    return FP8_OK;
}

// The bf16 operands' addresses (or'ed) and the steps' of a weight given as codes.
fp8_status_t check_aligned(const char* who, uintptr_t bf16, const float* steps) {
    if (bf16 & 1) return fail(FP8_EINVAL, "%s: a bf16 operand is not aligned to its elements", who);
    if ((uintptr_t)steps & 3)
        return fail(FP8_EINVAL, "%s: sw is not aligned to its elements", who);
    return FP8_OK;
}

fp8_status_t check_scratch(const char* who, const char* what, const void* p, size_t have,
                           size_t need) {
    if (need == 0) return FP8_OK;
    if (!p) return fail(FP8_EINVAL, "%s: %s is NULL", who, what);
    if (have < need) return fail(FP8_EINVAL, "%s: %s %zu < %zu bytes", who, what, have, need);
    if ((uintptr_t)p & 255) return fail(FP8_EINVAL, "%s: %s not 256-byte aligned", who, what);
    return FP8_OK;
}

fp8lin::BlockQuantLaunch quant_of(const uint16_t* x, int64_t rows, int64_t cols, fp8_fmt_t fmt,
                                  int32_t margin) {
    fp8lin::BlockQuantLaunch q;
    q.x = x;
    q.in_type = FP8_IN_BF16;
    q.rows = rows;
    q.cols = cols;
    q.ldx = cols;
    q.fmt = fmt;
    q.rmargin = ldexpf(1.0f, -margin);
    return q;
}

fp8lin::BlockGemmLaunch gemm_of(const uint8_t* a, const uint8_t* b, fp8_fmt_t fa, fp8_fmt_t fb,
                                int ta, int tb, int64_t m, int64_t n, int64_t k, const float* sa,
                                const float* sb, fp8_group_t group_b, const uint16_t* bias,
                                uint16_t* out) {
    fp8lin::BlockGemmLaunch g;
    g.a = a;
    g.b = b;
    g.fmt_a = fa;
    g.fmt_b = fb;
    g.trans_a = ta;
    g.trans_b = tb;
    g.m = m;
    g.n = n;
    g.k = k;
    g.lda = ta ? m : k;
    g.ldb = tb ? k : n;
    g.sa = scale_of(sa, FP8_GROUP_LINE, ta == 0, m, k);
    g.sb = scale_of(sb, group_b, tb != 0, n, k);
    g.bias = bias;
    g.out = out;
    return g;
}

}  // namespace

extern "C" {

size_t fp8_linear_block_saved(int64_t M, int64_t N, int64_t K, int32_t want_dx, int32_t want_dw) {
    if (M < 1 || N < 1 || K < 1) return 0;
    return saved_layout(M, N, K, want_dx != 0, want_dw != 0).total;
}
size_t fp8_linear_block_fwd_workspace(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || N < 1 || K < 1) return 0;
    return fwd_ws(M, N, K).total;
}
size_t fp8_linear_block_bwd_workspace(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || N < 1 || K < 1) return 0;
    return bwd_ws(M, N).total;
}

fp8_status_t fp8_linear_block_fwd(const uint16_t* x, const uint16_t* w, const uint8_t* w8,
                                  const float* sw, fp8_fmt_t fmt_w, const uint16_t* bias,
                                  int64_t M, int64_t N, int64_t K, fp8_fmt_t fmt, int32_t margin,
                                  void* saved, size_t saved_bytes, int32_t want_dx,
                                  int32_t want_dw, void* workspace, size_t workspace_bytes,
                                  uint16_t* out, hipStream_t stream) {
    clear_error();
    const char* who = "fp8_linear_block_fwd";
    if (!fmt_ok(fmt) || (w8 && !fmt_ok(fmt_w)))
        return fail(FP8_EINVAL, "%s: unsupported fp8 format", who);
    if (!x || !out) return fail(FP8_EINVAL, "%s: x or out is NULL", who);
    if ((w != nullptr) == (w8 != nullptr))
        return fail(FP8_EINVAL, "%s: the weight comes either as bf16 or as codes", who);
    if (w8 && !sw) return fail(FP8_EINVAL, "%s: codes of the weight need their steps", who);
    fp8_status_t st = check_layer(who, M, N, K, margin);
    if (st) return st;
    if ((st = check_aligned(who, (uintptr_t)x | (uintptr_t)w | (uintptr_t)bias | (uintptr_t)out,
                            w8 ? sw : nullptr)))
        return st;
    // a weight given as codes is its caller's to keep
    const SavedLayout S = saved_layout(M, N, K, want_dx && w, want_dw != 0);
    if ((st = check_scratch(who, "saved", saved, saved_bytes, S.total))) return st;
    const FwdWs L = fwd_ws(M, N, K);
    if ((st = check_scratch(who, "workspace", workspace, workspace_bytes, L.total))) return st;
    if ((st = check_device())) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint8_t* sv = static_cast<uint8_t*>(saved);
    fp8lin::BlockQuantLaunch qx = quant_of(x, M, K, fmt, margin);
    qx.out_row = ws + L.x8;
    qx.scale_row = reinterpret_cast<float*>(ws + L.sx);
    if (want_dw) {
        qx.out_col = sv + S.x8;
        qx.scale_col = reinterpret_cast<float*>(sv + S.sx);
    }
    hipError_t e;
    if (w) {
        uint8_t* at = want_dx ? sv + S.w8 : ws + L.w8;
        float* steps = reinterpret_cast<float*>(want_dx ? sv + S.sw : ws + L.sw);
        fp8lin::BlockQuantLaunch qw = quant_of(w, N, K, fmt, margin);
        qw.out_tile = at;
        qw.scale_tile = steps;
        e = fp8lin::launch_quantize_block_two(qx, qw, stream);
        w8 = at;
        sw = steps;
        fmt_w = fmt;
    } else {
        e = fp8lin::launch_quantize_block(qx, stream);
    }
    if (e != hipSuccess) return hip_fail(e, "block quantize launch");
    e = fp8lin::launch_block_gemm(gemm_of(qx.out_row, w8, fmt, fmt_w, 0, 1, M, N, K, qx.scale_row,
                                          sw, FP8_GROUP_TILE, bias, out), stream);
    return e == hipSuccess ? FP8_OK : hip_fail(e, "block gemm launch");
}

fp8_status_t fp8_linear_block_bwd(const uint16_t* g, const void* saved, size_t saved_bytes,
                                  const uint8_t* w8, const float* sw, fp8_fmt_t fmt_w, int64_t M,
                                  int64_t N, int64_t K, fp8_fmt_t fmt, fp8_fmt_t fmt_g,
                                  int32_t margin, int32_t want_dx, int32_t want_dw,
                                  void* workspace, size_t workspace_bytes, uint16_t* dx,
                                  uint16_t* dw, uint16_t* db, hipStream_t stream) {
    clear_error();
    const char* who = "fp8_linear_block_bwd";
    if (!fmt_ok(fmt) || !fmt_ok(fmt_g) || (w8 && !fmt_ok(fmt_w)))
        return fail(FP8_EINVAL, "%s: unsupported fp8 format", who);
    if (!g) return fail(FP8_EINVAL, "%s: g is NULL", who);
    if (w8 && !sw) return fail(FP8_EINVAL, "%s: codes of the weight need their steps", who);
    fp8_status_t st = check_layer(who, M, N, K, margin);
    if (st) return st;
    if ((st = check_aligned(who, (uintptr_t)g | (uintptr_t)dx | (uintptr_t)dw | (uintptr_t)db,
                            w8 ? sw : nullptr)))
        return st;
    if ((dx && !w8 && !want_dx) || (dw && !want_dw))
        return fail(FP8_EINVAL, "%s: a gradient whose codes the forward did not keep", who);
    const SavedLayout S = saved_layout(M, N, K, want_dx && !w8, want_dw != 0);
    if ((st = check_scratch(who, "saved", saved, saved_bytes, S.total))) return st;
    const BwdWs L = bwd_ws(M, N);
    if ((st = check_scratch(who, "workspace", workspace, workspace_bytes, L.total))) return st;
    if ((st = check_device())) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const uint8_t* sv = static_cast<const uint8_t*>(saved);
    hipError_t e = hipSuccess;
    fp8lin::ColsumFinalJob cf;
    fp8lin::BlockQuantLaunch q = quant_of(g, M, N, fmt_g, margin);
    if (dx) {
        q.out_row = ws + L.g8;
        q.scale_row = reinterpret_cast<float*>(ws + L.sg);
    }
    if (dw) {
        q.out_col = ws + L.g8c;
        q.scale_col = reinterpret_cast<float*>(ws + L.sgc);
    }
    if (db && dx && dw) {  // its partial sums come from the quantize's read of g
        q.sums = reinterpret_cast<float*>(ws + L.sums);
        cf.part = q.sums;
        cf.chunks = groups_of(M);
        cf.n = N;
        cf.db = db;
    } else if (db) {
        e = fp8lin::launch_colsum(g, M, N, db, ws + L.sums, stream);
        if (e != hipSuccess) return hip_fail(e, "colsum launch");
    }
    if (!dx && !dw) return FP8_OK;
    e = fp8lin::launch_quantize_block(q, stream);
    if (e != hipSuccess) return hip_fail(e, "block quantize launch");
    if (!w8) {
        w8 = sv + S.w8;
        sw = reinterpret_cast<const float*>(sv + S.sw);
        fmt_w = fmt;
    }
    // dX[M][K] = g8[M][N] . w8[N][K] (NN); dW[N][K] = g8c^T . x8c (TN)
    const fp8lin::BlockGemmLaunch gx = gemm_of(q.out_row, w8, fmt_g, fmt_w, 0, 0, M, K, N,
                                               q.scale_row, sw, FP8_GROUP_TILE, nullptr, dx);
    const fp8lin::BlockGemmLaunch gw =
        gemm_of(q.out_col, sv + S.x8, fmt_g, fmt, 1, 0, N, K, M, q.scale_col,
                reinterpret_cast<const float*>(sv + S.sx), FP8_GROUP_LINE, nullptr, dw);
    if (dx && dw) e = fp8lin::launch_block_gemm_pair(gx, gw, cf, stream);
    else e = fp8lin::launch_block_gemm(dx ? gx : gw, stream);
    return e == hipSuccess ? FP8_OK : hip_fail(e, "block gemm launch");
}

static const char* moe_sizes_error(int64_t tokens, int64_t experts, int64_t top_k, int64_t dim,
                                   int64_t hidden) {
    if (tokens < 0 || tokens > 1024) return "tokens outside [0, 1024]";
    if (experts < 1 || experts > 512) return "experts outside [1, 512]";
    if (top_k < 1 || top_k > 16 || top_k > experts) return "top_k outside [1, min(16, experts)]";
    if (dim < 16 || dim > 65536 || dim % 16) return "dim must be a multiple of 16 up to 65536";
    if (hidden < 16 || hidden > 65536 || hidden % 16)
        return "hidden must be a multiple of 16 up to 65536";
    return nullptr;
}

size_t fp8_moe_workspace(int64_t tokens, int64_t experts, int64_t top_k, int64_t dim,
                         int64_t hidden) {
    if (moe_sizes_error(tokens, experts, top_k, dim, hidden)) return 0;
    return fp8lin::moe_workspace(tokens, experts, top_k, dim, hidden);
}

fp8_status_t fp8_moe(const uint16_t* x, const uint16_t* router, const uint8_t* w13,
                     const float* s13, const uint8_t* w2, const float* s2, int64_t tokens,
                     int64_t experts, int64_t top_k, int64_t dim, int64_t hidden, fp8_fmt_t fmt,
                     int32_t renormalize, void* workspace, size_t workspace_bytes, uint16_t* out,
                     int32_t* ids, float* weights, hipStream_t stream) {
    clear_error();
    const char* who = "fp8_moe";
    if (!fmt_ok(fmt)) return fail(FP8_EINVAL, "%s: unsupported fp8 format %d", who, fmt);
    if (const char* why = moe_sizes_error(tokens, experts, top_k, dim, hidden))
        return fail(FP8_EINVAL, "%s: %s", who, why);
    if (tokens == 0) return FP8_OK;
    if (!x || !router || !w13 || !s13 || !w2 || !s2 || !workspace || !out)
        return fail(FP8_EINVAL, "%s: NULL operand, workspace or output", who);
    if (((uintptr_t)x | (uintptr_t)router | (uintptr_t)w13 | (uintptr_t)w2 | (uintptr_t)out) & 15)
        return fail(FP8_EINVAL, "%s: x, router, weights and out must be 16-byte aligned", who);
    if (((uintptr_t)s13 | (uintptr_t)s2 | (uintptr_t)ids | (uintptr_t)weights) & 3)
        return fail(FP8_EINVAL, "%s: steps, ids or weights not aligned to their elements", who);
    const size_t need = fp8lin::moe_workspace(tokens, experts, top_k, dim, hidden);
    if (workspace_bytes < need)
        return fail(FP8_EINVAL, "%s: workspace %zu < %zu bytes", who, workspace_bytes, need);
    if ((uintptr_t)workspace & 255)
        return fail(FP8_EINVAL, "%s: workspace not 256-byte aligned", who);
    fp8_status_t st = check_device();
    if (st) return st;
    fp8lin::MoeLaunch g;
    g.x = x;
    g.router = router;
    g.w13 = w13;
    g.s13 = s13;
    g.w2 = w2;
    g.s2 = s2;
    g.tokens = (int)tokens;
    g.experts = (int)experts;
    g.top_k = (int)top_k;
    g.dim = (int)dim;
    g.hidden = (int)hidden;
    g.fmt = fmt;
    g.renorm = renormalize != 0;
    g.ws = workspace;
    g.out = out;
    g.ids = ids;
    g.weights = weights;
    hipError_t e = fp8lin::launch_moe(g, stream);
    return e == hipSuccess ? FP8_OK : hip_fail(e, "mixture-of-experts launch");
}

}  // extern "C"
