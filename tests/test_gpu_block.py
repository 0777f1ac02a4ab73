"""Block-scaled operators on the GPU against plain 64-bit implementations
(tests/block_ref.py): codes and steps bit for bit, products and the
mixture-of-experts layer within bounds derived from their arithmetic."""

import numpy as np
import pytest
import torch

import workloads as wl
from tests import block_ref as ref
from tests.gpu_util import from_dev_bf16, from_dev_u8

pytestmark = pytest.mark.gpu

E4M3, E5M2 = 0, 1
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def f():
    import fp8_tensor_scaled_amd as f
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return f


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().float().cpu().numpy()


# --------------------------------------------------------------------------
# quantize
# --------------------------------------------------------------------------

def run_quantize(f, x, rows, cols, kinds, fmt, margin=0, ldx=None, stream=None):
    """{kind: (code bits, steps)}; buffers start with values no call leaves."""
    shape = {"row": (rows, ref.groups(cols)), "col": (ref.groups(rows), cols),
             "tile": (ref.groups(rows), ref.groups(cols))}
    kw, out = {}, {}
    for k in kinds:
        c = torch.full((rows * cols + 32,), 0xAB, dtype=torch.uint8, device="cuda")
        s = torch.full((shape[k][0] * shape[k][1] + 8,), -7.0, device="cuda")
        kw["out_" + k], kw["scale_" + k] = c, s
        out[k] = (c, s, shape[k])
    f.fp8_quantize_block(x, rows, cols, fmt, margin=margin, ldx=ldx, stream=stream, **kw)
    torch.cuda.synchronize()
    r = {}
    for k, (c, s, sh) in out.items():
        c, s = from_dev_u8(c), s.cpu().numpy()
        assert (c[rows * cols:] == 0xAB).all() and (s[sh[0] * sh[1]:] == -7.0).all(), "overrun"
        r[k] = (c[:rows * cols].reshape(rows, cols), s[:sh[0] * sh[1]].reshape(sh))
    return r


def check_quantize(f, x, kinds, fmt, margin=0, ldx=None, **kw):
    rows, cols = x.shape
    got = run_quantize(f, x, rows, cols, kinds, fmt, margin, ldx, **kw)
    v = host(x)
    for k, (codes, steps) in got.items():
        q, s = ref.quantize(v, k, fmt, margin)
        np.testing.assert_array_equal(steps, s, err_msg=f"{k} steps")
        np.testing.assert_array_equal(ref.decode(codes, fmt), q, err_msg=f"{k} codes")
    return got


KINDS = [("row",), ("col",), ("row", "col"), ("tile",)]


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (128, 1), (3, 129), (127, 255),
                                       (130, 264), (257, 1000), (16, 2048), (300, 7)])
def test_quantize_sizes(f, kinds, rows, cols):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((1, cols)))
    check_quantize(f, dev(x.astype(np.float32), torch.bfloat16), kinds, E4M3)


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("margin", [0, 3])
def test_quantize_types(f, fmt, dtype, margin):
    rng = np.random.default_rng(5)
    x = dev((rng.standard_normal((200, 392)) * 3e-3).astype(np.float32), DTYPES[dtype])
    for kinds in KINDS:
        check_quantize(f, x, kinds, fmt, margin)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("off,pad", [(0, 3), (1, 0), (5, 24), (8, 8)])
def test_quantize_strided_and_unaligned(f, dtype, off, pad):
    """Columns off .. off + 299 of a wider matrix: rows begin anywhere."""
    rng = np.random.default_rng(off)
    wide = dev(rng.standard_normal((150, off + 300 + pad)).astype(np.float32), DTYPES[dtype])
    x = wide[:, off:off + 300]
    for kinds in KINDS:
        check_quantize(f, x, kinds, E4M3, ldx=off + 300 + pad)


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_quantize_special_values(f, kinds, fmt):
    """All-zero groups, values below the smallest step, NaN, infinities, the
    type's largest value, subnormal inputs."""
    x = np.random.default_rng(9).standard_normal((260, 300)).astype(np.float32)
    x[:130, :140] = 0.0
    x[5, 200] = np.nan
    x[131, 10:20] = np.nan
    x[200, 290] = np.inf
    x[201, 150] = -np.inf
    x[250, 130:140] = 3.4e38
    x[140, 128:256] = 1e-20
    x[141, :128] = 1e-41
    x[259, :] = -0.0
    with np.errstate(all="ignore"):
        check_quantize(f, dev(x), kinds, fmt)


def test_quantize_empty(f):
    x = torch.empty(0, 200, dtype=torch.bfloat16, device="cuda")
    s = torch.full((8,), 3.0, device="cuda")
    f.fp8_quantize_block(x, 0, 200, E4M3, out_row=torch.empty(0, 200, dtype=torch.uint8,
                                                                 device="cuda"), scale_row=s)
    torch.cuda.synchronize()
    assert (s == 3.0).all()


def test_quantize_every_bf16(f):
    """Every finite bf16 value, one group a row: codes at every tie."""
    bits = np.arange(65536, dtype=np.uint32)
    v = (bits << 16).view(np.float32)
    v = np.where(np.isfinite(v), v, 0).reshape(512, 128)
    for fmt in (E4M3, E5M2):
        check_quantize(f, dev(v, torch.bfloat16), ("row", "col"), fmt)


# --------------------------------------------------------------------------
# product
# --------------------------------------------------------------------------

def run_mm(f, a, b, fa, fb, ta, tb, m, n, k, sa, ga, sb, gb, bias=None, lda=None, ldb=None,
           split=True, pad_out=64):
    out = torch.full((m * n + pad_out,), 0x7A11, dtype=torch.int16, device="cuda")
    need = f.fp8_mm_block_workspace(m, n, k) if split else 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
    lda = (m if ta else k) if lda is None else lda
    ldb = (k if tb else n) if ldb is None else ldb
    for _ in range(2):  # the second call finds the workspace as the first left it
        f.fp8_mm_block(a, b, fa, fb, ta, tb, m, n, k, lda, ldb, sa, ga, sb, gb, bias, out,
                       workspace=ws)
    torch.cuda.synchronize()
    o = from_dev_bf16(out)
    assert (o[m * n:] == 0x7A11).all(), "output overrun"
    return o[:m * n].reshape(m, n)


def operand(rows, cols, fmt, seed, ld=None):
    """Codes [rows][cols] in a buffer of row stride ld whose gaps hold NaN codes."""
    ld = cols if ld is None else ld
    buf = np.full((rows, ld), 0x7F, np.uint8)
    buf[:, :cols] = wl.random_codes((rows, cols), fmt, seed)
    return buf, ref.decode(buf[:, :cols], fmt)


def steps(shape, seed):
    r = np.random.default_rng(seed)
    return np.exp(r.standard_normal(shape)).astype(np.float32) * np.float32(0.01)


def check_mm(f, layout, m, n, k, fa=E4M3, fb=E4M3, tile_a=False, tile_b=True, bias=False, pad=0,
             split=True, seed=1):
    ta, tb = int(layout[0] == "t"), int(layout[1] == "t")
    ra, ca = (k, m) if ta else (m, k)
    rb, cb = (n, k) if tb else (k, n)
    abuf, av = operand(ra, ca, fa, seed, ca + pad)
    bbuf, bv = operand(rb, cb, fb, seed + 1, cb + pad)
    G = ref.groups

    def scales(rows, cols, trans_k, tile, sd):
        """(steps as stored, steps [line][kb]) for a stored [rows][cols]; trans_k: k runs down."""
        if tile:
            s = steps((G(rows), G(cols)), sd)
            full = np.repeat(s, 128, 1)[:, :cols] if trans_k else np.repeat(s, 128, 0)[:rows]
        else:
            s = steps((G(rows), cols) if trans_k else (rows, G(cols)), sd)
            full = s
        return s, (full.T if trans_k else full)

    sa, sav = scales(ra, ca, bool(ta), tile_a, seed + 2)
    sb, sbv = scales(rb, cb, not tb, tile_b, seed + 3)
    bias_bits = wl.normal_bf16((n,), 5.0, seed + 4) if bias else None
    value, bound = ref.product(av.T if ta else av, bv.T if tb else bv, sav, sbv.T,
                               wl.bf16_bits_to_f32(bias_bits).astype(float) if bias else None)
    got = run_mm(f, dev(abuf), dev(bbuf), fa, fb, ta, tb, m, n, k, dev(sa), int(tile_a), dev(sb),
                 int(tile_b), None if bias_bits is None else dev(bias_bits.view(np.int16)),
                 ca + pad, cb + pad, split)
    ref.check_close(got, value, bound, f"{layout} {m}x{n}x{k}")
    return got


@pytest.mark.parametrize("layout", ["nt", "nn", "tn", "tt"])
@pytest.mark.parametrize("tile_a,tile_b", [(False, True), (False, False), (True, False),
                                           (True, True)])
def test_mm_groupings(f, layout, tile_a, tile_b):
    check_mm(f, layout, 160, 208, 400, tile_a=tile_a, tile_b=tile_b, bias=True)


@pytest.mark.parametrize("layout", ["nt", "nn", "tn"])
@pytest.mark.parametrize("fa,fb", [(E4M3, E4M3), (E5M2, E4M3), (E5M2, E5M2), (E4M3, E5M2)])
def test_mm_formats(f, layout, fa, fb):
    check_mm(f, layout, 144, 272, 272, fa, fb, tile_b=layout != "tn")


@pytest.mark.parametrize("layout", ["nt", "nn", "tn"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 128, 128), (5, 3, 129), (17, 33, 127),
                                   (64, 256, 1024), (65, 130, 257), (130, 129, 640),
                                   (256, 384, 144), (300, 272, 528)])
@pytest.mark.parametrize("tile_b", [True, False])
def test_mm_sizes(f, layout, m, n, k, tile_b):
    check_mm(f, layout, m, n, k, tile_b=tile_b, bias=(m + n + k) % 2 == 1)


@pytest.mark.parametrize("layout", ["nt", "nn", "tn", "tt"])
@pytest.mark.parametrize("pad", [1, 3, 8, 16])
def test_mm_row_strides(f, layout, pad):
    check_mm(f, layout, 96, 160, 304, pad=pad)


@pytest.mark.parametrize("m", [1, 2, 7, 16, 17, 33, 64])
@pytest.mark.parametrize("n,k", [(256, 4096), (48, 8192), (1000, 1040)])
def test_mm_few_rows(f, m, n, k):
    """Short A, long k: the products that may be split along k, with and
    without the workspace that allows it."""
    check_mm(f, "nt", m, n, k, split=True, bias=True)
    check_mm(f, "nt", m, n, k, split=False, bias=True)


def test_mm_sums_in_a_fixed_order(f):
    for args in (("nt", 16, 256, 4096), ("nt", 300, 272, 528), ("tn", 144, 160, 400)):
        a = check_mm(f, *args, tile_b=args[0] != "tn")
        b = check_mm(f, *args, tile_b=args[0] != "tn")
        assert np.array_equal(a, b)


def sampled_product(f, layout, m, n, k, fa, fb, tile_b, bias, rows=24, cols=24):
    """A large product, checked on the corners, tile borders and random rows x columns."""
    ta, tb = int(layout[0] == "t"), int(layout[1] == "t")
    rng = np.random.default_rng(m + n + k)
    pick = lambda hi, c: np.unique(np.concatenate([  # noqa: E731
        [0, hi - 1, hi // 2], np.minimum(hi - 1, [127, 128, 255, 256]), rng.integers(0, hi, c)]))
    ri, ci = pick(m, rows), pick(n, cols)
    shape_a, shape_b = ((k, m) if ta else (m, k)), ((n, k) if tb else (k, n))
    a, b = wl.random_codes(shape_a, fa, 11), wl.random_codes(shape_b, fb, 12)
    G = ref.groups
    sa = steps((G(k), m) if ta else (m, G(k)), 13)
    sb = steps(((G(n), G(k)) if tb else (G(k), G(n))) if tile_b else
               ((n, G(k)) if tb else (G(k), n)), 14)
    bias_bits = wl.normal_bf16((n,), 5.0, 15) if bias else None
    got = run_mm(f, dev(a), dev(b), fa, fb, ta, tb, m, n, k, dev(sa), 0, dev(sb), int(tile_b),
                 None if bias_bits is None else dev(bias_bits.view(np.int16)))
    av = ref.decode(a[:, ri].T if ta else a[ri], fa)
    bv = ref.decode(b[ci].T if tb else b[:, ci], fb)
    sav = sa[:, ri].T if ta else sa[ri]
    cg = ci // 128 if tile_b else ci
    sbv = sb[cg].T if tb else sb[:, cg]
    value, bound = ref.product(av, bv, sav, sbv, wl.bf16_bits_to_f32(bias_bits[ci]).astype(float)
                               if bias else None)
    ref.check_close(got[np.ix_(ri, ci)], value, bound, f"{layout} {m}x{n}x{k}")
    y = wl.bf16_bits_to_f32(got)
    assert np.isfinite(y).all()


@pytest.mark.parametrize("layout,m,n,k,fa,fb,tile_b,bias", [
    ("nt", 4096, 4096, 512, E4M3, E4M3, True, True),
    ("nt", 2064, 4112, 272, E4M3, E4M3, True, True),
    ("nt", 2048, 2048, 384, E4M3, E4M3, False, False),
    ("nn", 2048, 1024, 1024, E5M2, E4M3, True, False),
    ("nn", 3000, 1040, 400, E5M2, E5M2, True, False),
    ("nn", 1024, 2048, 384, E4M3, E4M3, False, False),
    ("tn", 4096, 1024, 512, E5M2, E4M3, False, False),
    ("tn", 2064, 2080, 400, E4M3, E4M3, False, False),
    ("tn", 1040, 4096, 384, E4M3, E4M3, True, False),
    ("nt", 1111, 2001, 777, E4M3, E4M3, True, True),
    ("nn", 1000, 1111, 2047, E5M2, E4M3, True, False),
    ("tn", 1003, 999, 601, E5M2, E4M3, False, False),
    ("nt", 64, 8192, 2048, E4M3, E4M3, True, False),
])
def test_mm_large(f, layout, m, n, k, fa, fb, tile_b, bias):
    sampled_product(f, layout, m, n, k, fa, fb, tile_b, bias)


def test_mm_special_codes(f):
    """A NaN code reaches its own row (column) only; infinities of E5M2 stay."""
    m, n, k = 48, 160, 272
    a, b = wl.random_codes((m, k), E5M2, 3), wl.random_codes((n, k), E4M3, 4)
    b[:, 40] = 0x38  # 1.0
    a[7, 40] = 0x7C  # +inf
    a[9, 100] = 0x7E  # NaN
    b[5, 200] = 0x7F  # NaN
    got = wl.bf16_bits_to_f32(run_mm(f, dev(a), dev(b), E5M2, E4M3, 0, 1, m, n, k,
                                     dev(steps((m, 3), 1)), 0, dev(steps((2, 3), 2)), 1))
    ok = np.ones((m, n), bool)
    ok[7] = ok[9] = False
    ok[:, 5] = False
    assert np.isfinite(got[ok]).all()
    assert np.isnan(got[9]).all() and np.isnan(got[:, 5]).all()
    assert np.isposinf(np.delete(got[7], 5)).all()


# --------------------------------------------------------------------------
# layer
# --------------------------------------------------------------------------

@pytest.fixture(scope="module")
def ac(f):
    from fp8_tensor_scaled_amd import autocast
    return autocast


def layer_reference(x, w, bias, g, ff, fb, margin=0):
    """Values and bounds of y, dx, dw, db from the definitions."""
    q = lambda v, kind, fmt: ref.quantize(v, kind, fmt, margin)  # noqa: E731
    (xr, sxr), (xc, sxc) = q(x, "row", ff), q(x, "col", ff)
    (gr, sgr), (gc, sgc) = q(g, "row", fb), q(g, "col", fb)
    wq, sw = q(w, "tile", ff)
    n, k = w.shape
    y = ref.product(xr, wq.T, sxr, np.repeat(sw, 128, 0)[:n].T, bias)
    dx = ref.product(gr, wq, sgr, np.repeat(sw, 128, 1)[:, :k])
    dw = ref.product(gc.T, xc, sgc.T, sxc)
    m = g.shape[0]
    db = (g.astype(float).sum(0), m * 2.0 ** -24 * np.abs(g.astype(float)).sum(0))
    return y, dx, dw, db


@pytest.mark.parametrize("fmt", ["hybrid", "e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K,bias,margin", [(160, 272, 400, True, 0), (1, 128, 256, False, 0),
                                               (33, 130, 70, True, 2), (256, 256, 256, True, 0)])
def test_layer(f, ac, fmt, M, N, K, bias, margin):
    rng = np.random.default_rng(M + N)
    b16 = lambda *s, std=1.0: wl.f32_to_bf16_bits(rng.standard_normal(s) * std)  # noqa: E731
    t = lambda h: dev(h.view(np.int16)).view(torch.bfloat16)  # noqa: E731
    xb, wb, gb, bb = b16(M, K), b16(N, K, std=0.02), b16(M, N, std=1e-3), b16(N)
    x, w = t(xb).requires_grad_(True), t(wb).requires_grad_(True)
    b = t(bb).requires_grad_(True) if bias else None
    with ac.fp8_autocast(recipe=ac.FP8Recipe(block=True, margin=margin), fp8_format=fmt):
        y = ac.fp8_linear(x, w, b)
    y.backward(t(gb))
    torch.cuda.synchronize()
    v = wl.bf16_bits_to_f32
    F = ac.FP8Format(fmt)
    want = layer_reference(v(xb), v(wb), v(bb).astype(float) if bias else None, v(gb), F.fwd(),
                           F.bwd(), margin)
    bits = lambda a: from_dev_bf16(a.detach().view(torch.int16))  # noqa: E731
    for got, (value, bound), what in zip((y, x.grad, w.grad, b.grad if bias else None), want,
                                         ("y", "dx", "dw", "db")):
        if got is not None:
            ref.check_close(bits(got), value, bound, f"{fmt} {what}")


def test_layer_gradient_against_differences(f, ac):
    """Along random directions the loss changes by what the gradients say, up
    to the codes' own rounding: with values that the codes hold exactly."""
    rng = np.random.default_rng(2)
    M, N, K = 48, 128, 256
    small = lambda *s: rng.integers(-7, 8, s).astype(np.float32)  # noqa: E731
    x, w, g = small(M, K), small(N, K), small(M, N)
    # every group's largest magnitude is 7 = 448 / 64, so steps are powers of two and codes exact
    x[:, ::64] = 7
    w[::64, ::64] = 7
    g[:, ::64] = 7
    x[::32] = 7
    g[::32] = 7
    t = lambda a: dev(a, torch.bfloat16)  # noqa: E731
    xt, wt = t(x).requires_grad_(True), t(w).requires_grad_(True)
    with ac.fp8_autocast(recipe=ac.FP8Recipe(block=True), fp8_format="e4m3"):
        ac.fp8_linear(xt, wt).backward(t(g))
    gx, gw = host(xt.grad).astype(float), host(wt.grad).astype(float)
    x, w, g = (v.astype(float) for v in (x, w, g))
    loss = lambda a, b: float((a @ b.T * g).sum())  # noqa: E731
    for _ in range(4):
        ux, uw = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        h = 1e-3
        dx = (loss(x + h * ux, w) - loss(x - h * ux, w)) / (2 * h)
        dw = (loss(x, w + h * uw) - loss(x, w - h * uw)) / (2 * h)
        # each gradient is a bf16 rounding (2^-9) of the exact one
        assert abs((gx * ux).sum() - dx) <= 2.0 ** -8 * np.abs(gx * ux).sum()
        assert abs((gw * uw).sum() - dw) <= 2.0 ** -8 * np.abs(gw * uw).sum()


def test_layer_partial_gradients_and_shapes(f, ac):
    x = torch.randn(2, 3, 5, 144, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(96, 144, device="cuda", dtype=torch.bfloat16)
    g = torch.randn(2, 3, 5, 96, device="cuda", dtype=torch.bfloat16)
    recipe = ac.FP8Recipe(block=True)
    full = {}
    for need in ((1, 1), (1, 0), (0, 1)):
        xi, wi = x.clone().requires_grad_(bool(need[0])), w.clone().requires_grad_(bool(need[1]))
        with ac.fp8_autocast(recipe=recipe):
            y = ac.fp8_linear(xi, wi)
        assert y.shape == (2, 3, 5, 96)
        y.backward(g)
        for name, a in (("x", xi), ("w", wi)):
            if a.requires_grad:
                assert a.grad.shape == a.shape
                assert torch.equal(full.setdefault(name, a.grad), a.grad)
    with torch.no_grad(), ac.fp8_autocast(recipe=recipe):
        assert torch.equal(ac.fp8_linear(x, w), y.detach())
    # a transposed (non-contiguous) input and gradient
    xt = x.reshape(30, 144).t().contiguous().t().requires_grad_(True)
    with ac.fp8_autocast(recipe=recipe):
        yt = ac.fp8_linear(xt, w)
    yt.backward(g.reshape(30, 96).t().contiguous().t())
    assert torch.equal(yt.reshape(y.shape), y.detach())
    assert torch.equal(xt.grad.reshape(x.shape), full["x"])


@pytest.mark.parametrize("M,N,K", [(2048, 2816, 2064), (2048, 2056, 2048)])
def test_layer_backward_beyond_one_launch(f, M, N, K):
    """Too many tiles for one launch of both products, and sides that the
    tiled kernels do not take: the bits of the products called one by one."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    x, w, dy = r(M, K), r(N, K), r(M, N)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    saved = u8(f.fp8_linear_block_saved(M, N, K, True, True))
    y, dx, dw = (torch.empty(*s, dtype=torch.bfloat16, device="cuda")
                 for s in ((M, N), (M, K), (N, K)))
    db = torch.empty(N, dtype=torch.bfloat16, device="cuda")
    zeros = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    f.fp8_linear_block_fwd(x, w, None, M, N, K, E4M3, 0, saved, True, True,
                           zeros(f.fp8_linear_block_fwd_workspace(M, N, K)), y)
    f.fp8_linear_block_bwd(dy, saved, M, N, K, E4M3, E5M2, 0, True, True,
                           zeros(f.fp8_linear_block_bwd_workspace(M, N, K)), dx, dw, db)
    G = ref.groups
    step = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    xr, xc, sxr, sxc = u8(M, K), u8(M, K), step(M, G(K)), step(G(M), K)
    gr, gc, sgr, sgc = u8(M, N), u8(M, N), step(M, G(N)), step(G(M), N)
    wt, sw = u8(N, K), step(G(N), G(K))
    f.fp8_quantize_block(x, M, K, E4M3, out_row=xr, scale_row=sxr, out_col=xc, scale_col=sxc)
    f.fp8_quantize_block(dy, M, N, E5M2, out_row=gr, scale_row=sgr, out_col=gc, scale_col=sgc)
    f.fp8_quantize_block(w, N, K, E4M3, out_tile=wt, scale_tile=sw)
    y1, dx1, dw1 = (torch.empty_like(t) for t in (y, dx, dw))
    f.fp8_mm_block(xr, wt, E4M3, E4M3, 0, 1, M, N, K, K, K, sxr, f.GROUP_LINE, sw, f.GROUP_TILE,
                   None, y1)
    f.fp8_mm_block(gr, wt, E5M2, E4M3, 0, 0, M, K, N, N, K, sgr, f.GROUP_LINE, sw, f.GROUP_TILE,
                   None, dx1)
    f.fp8_mm_block(gc, xc, E5M2, E4M3, 1, 0, N, K, M, N, K, sgc, f.GROUP_LINE, sxc, f.GROUP_LINE,
                   None, dw1)
    torch.cuda.synchronize()
    for a, b in ((y, y1), (dx, dx1), (dw, dw1)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    want = host(dy).astype(np.float64).sum(0)
    mag = np.abs(host(dy)).astype(np.float64).sum(0)
    ref.check_close(from_dev_bf16(db.view(torch.int16)), want, M * 2.0 ** -24 * mag, "db")


def test_layer_no_rows(f, ac):
    x = torch.empty(0, 144, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    w = torch.randn(96, 144, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    b = torch.randn(96, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    with ac.fp8_autocast(recipe=ac.FP8Recipe(block=True)):
        y = ac.fp8_linear(x, w, b)
    assert y.shape == (0, 96)
    y.backward(torch.empty(0, 96, device="cuda", dtype=torch.bfloat16))
    assert x.grad.shape == (0, 144) and not w.grad.any() and not b.grad.any()


def test_layer_weight_codes(f, ac):
    """A weight given as codes with tile steps: the bits of quantizing it here."""
    x = torch.randn(20, 272, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(144, 272, device="cuda", dtype=torch.bfloat16) * 0.02
    b = torch.randn(144, device="cuda", dtype=torch.bfloat16)
    w8 = torch.empty(144, 272, dtype=torch.float8_e4m3fn, device="cuda")
    sw = torch.empty(2, 3, device="cuda")
    f.fp8_quantize_block(w, 144, 272, E4M3, out_tile=w8, scale_tile=sw)
    g = torch.randn(20, 144, device="cuda", dtype=torch.bfloat16)
    grads = []
    for weight, scale in ((w, None), (w8, sw)):
        xi, bi = x.clone().requires_grad_(True), b.clone().requires_grad_(True)
        with ac.fp8_autocast(recipe=ac.FP8Recipe(block=True)):
            y = ac.fp8_linear(xi, weight, bi, w_scale=scale)
        y.backward(g)
        grads.append((y.detach(), xi.grad, bi.grad))
    for a, c in zip(*grads):
        assert torch.equal(a, c)


# --------------------------------------------------------------------------
# mixture of experts
# --------------------------------------------------------------------------

def moe_inputs(t, e, d, h, fmt, seed, wstd=1.0):
    G = ref.groups
    x = wl.normal_bf16((t, d), 1.0, seed)
    r = wl.normal_bf16((e, d), 1.5 / np.sqrt(d), seed + 1)
    w13 = wl.random_codes((e, 2 * h, d), fmt, seed + 2)
    w2 = wl.random_codes((e, d, h), fmt, seed + 3)
    spread = 448 / 6 if fmt == 0 else 57344 / 16
    s13 = steps((e, G(2 * h), G(d)), seed + 4) * np.float32(100 * wstd / spread / np.sqrt(d))
    s2 = steps((e, G(d), G(h)), seed + 5) * np.float32(100 * wstd / spread / np.sqrt(h))
    return x, r, w13, s13.astype(np.float32), w2, s2.astype(np.float32)


def moe_device(f, ins, t, e, k, d, h, fmt, renorm, ws=None, stream=None):
    x, r, w13, s13, w2, s2 = ins
    need = f.fp8_moe_workspace(t, e, k, d, h)
    if ws is None:
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    out = torch.full((t * d + 64,), 0x7A11, dtype=torch.int16, device="cuda")
    ids = torch.full((t * k + 8,), -9, dtype=torch.int32, device="cuda")
    wt = torch.full((t * k + 8,), -9.0, device="cuda")
    args = [dev(x.view(np.int16)), dev(r.view(np.int16)), dev(w13), dev(s13), dev(w2), dev(s2)]
    for _ in range(2):  # the second call finds the workspace as the first left it
        f.fp8_moe(*args, t, e, k, d, h, fmt, renorm, ws, out, ids=ids, weights=wt)
    torch.cuda.synchronize()
    o, i, w = from_dev_bf16(out), ids.cpu().numpy(), wt.cpu().numpy()
    assert (o[t * d:] == 0x7A11).all() and (i[t * k:] == -9).all() and (w[t * k:] == -9).all()
    return o[:t * d].reshape(t, d), i[:t * k].reshape(t, k), w[:t * k].reshape(t, k)


def moe_values(ins, e, d, h, fmt):
    x, r, w13, s13, w2, s2 = ins
    w13v = np.stack([ref.decode(w13[i], fmt) * ref.grow(s13[i], 2 * h, d, 128, 128)
                     for i in range(e)])
    w2v = np.stack([ref.decode(w2[i], fmt) * ref.grow(s2[i], d, h, 128, 128) for i in range(e)])
    v = lambda b: wl.bf16_bits_to_f32(b).astype(np.float64)  # noqa: E731
    return v(x), v(r), w13v, w2v


def check_moe(f, t, e, k, d, h, fmt=E4M3, renorm=True, seed=21, ins=None, ws=None):
    ins = moe_inputs(t, e, d, h, fmt, seed) if ins is None else ins
    got, ids, wt = moe_device(f, ins, t, e, k, d, h, fmt, renorm, ws)
    xv, rv, w13v, w2v = moe_values(ins, e, d, h, fmt)
    out, bound, wids, ww = ref.moe(xv, rv, w13v, w2v, k, renorm)
    np.testing.assert_array_equal(ids, wids)
    np.testing.assert_allclose(wt, ww, rtol=2e-5, atol=1e-30)
    ref.check_close(got, out, bound, f"moe {t} {e} {k} {d} {h}")
    return got


@pytest.mark.parametrize("t,e,k,d,h", [
    (1, 1, 1, 16, 16), (1, 8, 2, 128, 128), (1, 64, 8, 512, 256), (2, 4, 4, 144, 48),
    (3, 65, 6, 256, 144), (13, 32, 2, 272, 176), (16, 8, 1, 384, 128), (17, 8, 2, 256, 208),
    (33, 4, 2, 160, 160), (64, 16, 8, 256, 128), (70, 3, 2, 128, 272), (5, 300, 16, 128, 64)])
def test_moe_sizes(f, t, e, k, d, h):
    check_moe(f, t, e, k, d, h, renorm=(t + k) % 2 == 0)


@pytest.mark.parametrize("e,k,d,h", [(16, 16, 64, 2064), (16, 9, 48, 16), (12, 5, 272, 144),
                                     (130, 3, 16, 640), (512, 1, 80, 48), (4, 2, 128, 4096),
                                     (70, 8, 2048, 256)])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_moe_one_token(f, e, k, d, h, fmt):
    check_moe(f, 1, e, k, d, h, fmt=fmt, renorm=k % 2 == 1, seed=e + k)


def test_moe_one_token_ties_and_nan(f):
    e, k, d, h = 70, 4, 128, 32
    ins = list(moe_inputs(1, e, d, h, E4M3, 5))
    ins[1] = np.zeros_like(ins[1])  # every logit is 0
    _, ids, _ = moe_device(f, ins, 1, e, k, d, h, E4M3, True)
    assert (ids == np.arange(k)).all()
    ins[0] = np.full_like(ins[0], 0x7FC0)  # a NaN token
    got, ids, wt = moe_device(f, ins, 1, e, k, d, h, E4M3, True)
    assert np.isnan(wl.bf16_bits_to_f32(got)).all() and np.isnan(wt).all()
    assert (ids == np.arange(k)).all()


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("renorm", [True, False])
def test_moe_formats(f, fmt, renorm):
    check_moe(f, 9, 12, 3, 272, 144, fmt=fmt, renorm=renorm)


@pytest.mark.parametrize("t", [130, 200])
def test_moe_one_expert_takes_every_token(f, t):
    """All tokens choose the same two experts: lists far beyond one tile of tokens."""
    d, h, e = 128, 144, 6
    ins = list(moe_inputs(t, e, d, h, E4M3, 5))
    x = np.abs(wl.bf16_bits_to_f32(ins[0]))
    ins[0] = wl.f32_to_bf16_bits(x)
    r = np.zeros((e, d), np.float32)
    r[4], r[1] = 0.5, 0.25
    ins[1] = wl.f32_to_bf16_bits(r)
    got = check_moe(f, t, e, 2, d, h, ins=tuple(ins))
    assert got.shape == (t, d)


def test_moe_ties_go_to_the_lowest_index(f):
    t, e, k, d, h = 5, 70, 4, 128, 32
    ins = list(moe_inputs(t, e, d, h, E4M3, 6))
    r = wl.bf16_bits_to_f32(ins[1]).copy()
    r[3] = r[66] = r[20] = r[64]
    r[10] = r[11]
    ins[1] = wl.f32_to_bf16_bits(r)
    check_moe(f, t, e, k, d, h, ins=tuple(ins))
    ins[1] = np.zeros_like(ins[1])  # every logit equal
    _, ids, wt = moe_device(f, tuple(ins), t, e, k, d, h, E4M3, True)
    assert (ids == np.arange(k)).all() and np.allclose(wt, 1 / k, rtol=1e-6)


def test_moe_nan_and_infinite_tokens(f):
    """A token whose logits are NaN gets NaN and keeps it to itself."""
    t, e, k, d, h = 6, 16, 3, 144, 48
    ins = list(moe_inputs(t, e, d, h, E4M3, 7))
    clean = check_moe(f, t, e, k, d, h, ins=tuple(ins))
    x = ins[0].copy()
    x[2, 5] = 0x7FC0  # NaN
    x[4, 0] = 0x7F80  # +inf
    ins[0] = x
    got, ids, _ = moe_device(f, tuple(ins), t, e, k, d, h, E4M3, True)
    keep = [0, 1, 3, 5]
    assert np.array_equal(got[keep], clean[keep])
    y = wl.bf16_bits_to_f32(got)
    assert np.isnan(y[2]).all() and not np.isfinite(y[4]).any()
    assert ((0 <= ids) & (ids < e)).all()
    assert all(len(set(row)) == k for row in ids)


def test_moe_large_activations(f):
    """Gates far on either side: silu saturates without overflow or NaN."""
    t, e, k, d, h = 4, 4, 2, 128, 64
    ins = list(moe_inputs(t, e, d, h, E4M3, 8, wstd=200.0))
    got = check_moe(f, t, e, k, d, h, ins=tuple(ins))
    assert np.isfinite(wl.bf16_bits_to_f32(got)).all()


def test_moe_workspace_serves_other_shapes(f):
    shapes = [(9, 12, 3, 272, 144), (1, 64, 8, 512, 256), (40, 6, 2, 128, 64)]
    need = max(f.fp8_moe_workspace(*s) for s in shapes)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for s in shapes + shapes[::-1]:
        check_moe(f, *s, ws=ws)


def test_moe_same_bits_every_time(f):
    a = check_moe(f, 21, 12, 4, 272, 144)
    for _ in range(3):
        assert np.array_equal(a, check_moe(f, 21, 12, 4, 272, 144))


# --------------------------------------------------------------------------
# streams and graphs
# --------------------------------------------------------------------------

def test_other_streams(f):
    """Calls on a stream of the user's, ordered there after the inputs' making."""
    s = torch.cuda.Stream()
    rng = np.random.default_rng(4)
    xn = rng.standard_normal((200, 300)).astype(np.float32)
    with torch.cuda.stream(s):
        x = dev(xn, torch.bfloat16)
        got = run_quantize(f, x, 200, 300, ("row",), E4M3)
    q, st = ref.quantize(host(x), "row", E4M3)
    assert np.array_equal(ref.decode(got["row"][0], E4M3), q) and np.array_equal(got["row"][1], st)
    x = dev(xn, torch.bfloat16)
    torch.cuda.synchronize()
    got = run_quantize(f, x, 200, 300, ("row",), E4M3, stream=s)
    assert np.array_equal(got["row"][1], st)


def test_graph_replays(f):
    """One captured quantize, product and layer of experts; every replay on
    new inputs gives the eager call's bits, with eager work between."""
    t, e, k, d, h = 7, 12, 3, 256, 144
    x0, r, w13, s13, w2, s2 = moe_inputs(t, e, d, h, E4M3, 31)
    args = [dev(a.view(np.int16)) if a.dtype == np.uint16 else dev(a)
            for a in (r, w13, s13, w2, s2)]
    x = dev(x0.view(np.int16)).view(torch.bfloat16).reshape(t, d)
    wd = torch.randn(320, d, device="cuda", dtype=torch.bfloat16)
    w8 = torch.empty(320, d, dtype=torch.uint8, device="cuda")
    sw = torch.empty(3, 2, device="cuda")
    f.fp8_quantize_block(wd, 320, d, E4M3, out_tile=w8, scale_tile=sw)

    def buffers():
        need = f.fp8_mm_block_workspace(t, 320, d)
        return dict(x8=torch.empty(t, d, dtype=torch.uint8, device="cuda"),
                    sx=torch.empty(t, 2, device="cuda"),
                    y=torch.empty(t, 320, dtype=torch.bfloat16, device="cuda"),
                    ws=torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None,
                    mws=torch.zeros(f.fp8_moe_workspace(t, e, k, d, h), dtype=torch.uint8,
                                    device="cuda"),
                    out=torch.empty(t, d, dtype=torch.bfloat16, device="cuda"),
                    ids=torch.empty(t, k, dtype=torch.int32, device="cuda"))

    def calls(b):
        f.fp8_quantize_block(x, t, d, E4M3, out_row=b["x8"], scale_row=b["sx"])
        f.fp8_mm_block(b["x8"], w8, E4M3, E4M3, 0, 1, t, 320, d, d, d, b["sx"], f.GROUP_LINE, sw,
                       f.GROUP_TILE, None, b["y"], workspace=b["ws"])
        f.fp8_moe(x, args[0], args[1], args[2], args[3], args[4], t, e, k, d, h, E4M3, True,
                  b["mws"], b["out"], ids=b["ids"])

    eager, graphed = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(graphed)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(graphed)
    for i in range(4):
        x.copy_(torch.randn(t, d, device="cuda"))
        calls(eager)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for name in ("x8", "sx", "y", "out", "ids"):
            assert torch.equal(eager[name], graphed[name]), (i, name)
