"""The block quantize from 512 tiles on, and the expert layer from 1024
workgroups a product on, where both take another form than for less."""

import numpy as np
import pytest
import torch

import workloads as wl
from tests import block_ref as ref
from tests import block_ref_gpu as gref
from tests.gpu_util import from_dev_bf16, from_dev_u8

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
KINDS = [("row",), ("col",), ("row", "col"), ("tile",)]


@pytest.fixture(scope="module")
def f():
    import fp8_tensor_scaled_amd as f
    return f


def check_quantize(f, x, kinds, fmt, margin=0):
    rows, cols = x.shape
    assert ref.groups(rows) * ref.groups(cols) >= 512
    shape = {"row": (rows, ref.groups(cols)), "col": (ref.groups(rows), cols),
             "tile": (ref.groups(rows), ref.groups(cols))}
    kw, got = {}, {}
    for kind in kinds:
        c = torch.full((rows * cols + 32,), 0xAB, dtype=torch.uint8, device="cuda")
        s = torch.full((shape[kind][0] * shape[kind][1] + 8,), -7.0, device="cuda")
        kw["out_" + kind], kw["scale_" + kind], got[kind] = c, s, (c, s)
    f.fp8_quantize_block(x, rows, cols, fmt, margin=margin, ldx=x.stride(0), **kw)
    torch.cuda.synchronize()
    v = x.float().cpu().numpy()
    for kind, (c, s) in got.items():
        q, want = ref.quantize(v, kind, fmt, margin)
        c, s = from_dev_u8(c), s.cpu().numpy()
        assert (c[rows * cols:] == 0xAB).all() and (s[want.size:] == -7.0).all(), "overrun"
        np.testing.assert_array_equal(s[:want.size].reshape(want.shape), want, err_msg=kind)
        np.testing.assert_array_equal(ref.decode(c[:rows * cols].reshape(rows, cols), fmt), q,
                                      err_msg=kind)


def values(rows, cols, dtype, seed):
    """A strided slice, its columns of different sizes, its first element anywhere."""
    g = gref.generator(seed)
    wide = torch.randn(rows, cols + 11, device="cuda", generator=g)
    wide *= torch.exp(torch.randn(1, cols + 11, device="cuda", generator=g))
    return wide.to(DTYPES[dtype])[:, 3:3 + cols]


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(65500, 7), (9, 65501), (1927, 4351)])
def test_quantize(f, rows, cols, dtype, fmt, kinds):
    check_quantize(f, values(rows, cols, dtype, rows + fmt), kinds, fmt)


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_quantize_whole_rows(f, dtype, kinds):
    """Contiguous rows of whole 8s (codes go out 8 at a time), with a margin."""
    x = values(2056, 4104, dtype, 5).contiguous()
    check_quantize(f, x, kinds, E4M3, margin=2)
    check_quantize(f, x, kinds, E4M3)


@pytest.mark.parametrize("kinds", KINDS)
def test_quantize_special_values(f, kinds):
    x = values(2000, 4300, "f32", 6).contiguous()
    x[:130, :140] = 0.0
    x[5, 200], x[131, 10:20] = float("nan"), float("nan")
    x[1900, 4290], x[201, 150] = float("inf"), -float("inf")
    x[250, 130:140], x[140, 128:256], x[141, :128] = 3.4e38, 1e-20, 1e-41
    x[1999] = -0.0
    with np.errstate(all="ignore"):
        check_quantize(f, x, kinds, E4M3)


@pytest.mark.parametrize("fmt,fmt_g", [(E4M3, E5M2), (E4M3, E4M3), (E5M2, E5M2)])
@pytest.mark.parametrize("M,N,K", [(8200, 1032, 144), (4104, 272, 2064), (2063, 4111, 130)])
def test_layer(f, M, N, K, fmt, fmt_g):
    """A layer whose x or g has so many tiles: with and without the codes for
    the weight gradient, the bias gradient from g's quantize and by itself."""
    assert max(ref.groups(M) * ref.groups(N), ref.groups(M) * ref.groups(K)) >= 512
    r = lambda *s, seed: torch.randn(*s, device="cuda",  # noqa: E731
                                     generator=gref.generator(seed)).bfloat16()
    x, w, dy = r(M, K, seed=1), r(N, K, seed=2), r(M, N, seed=3)
    buf = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    b16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    fws = buf(f.fp8_linear_block_fwd_workspace(M, N, K))
    bws = buf(f.fp8_linear_block_bwd_workspace(M, N, K))
    q = lambda t, ft, kind: ref.quantize(t.float().cpu().numpy(), kind, ft)  # noqa: E731
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    wq, sw = (dev(a) for a in q(w, fmt, "tile"))
    xr, sxr = (dev(a) for a in q(x, fmt, "row"))
    xc, sxc = (dev(a) for a in q(x, fmt, "col"))
    gr, sgr = (dev(a) for a in q(dy, fmt_g, "row"))
    gc, sgc = (dev(a) for a in q(dy, fmt_g, "col"))
    want = dict(
        y=gref.product(xr, wq.t(), sxr, sw.repeat_interleave(128, 0)[:N].t()),
        dx=gref.product(gr, wq, sgr, sw.repeat_interleave(128, 1)[:, :K]),
        dw=gref.product(gc.t(), xc, sgc.t(), sxc),
        db=(dy.double().sum(0), M * 2.0 ** -24 * dy.double().abs().sum(0)))
    for need in (("dx", "dw", "db"), ("dx", "db"), ("dw",)):
        wx, ww = "dx" in need, "dw" in need
        saved = buf(f.fp8_linear_block_saved(M, N, K, wx, ww))
        got = dict(y=b16(M, N), dx=b16(M, K), dw=b16(N, K), db=b16(N))
        f.fp8_linear_block_fwd(x, w, None, M, N, K, fmt, 0, saved, wx, ww, fws, got["y"])
        f.fp8_linear_block_bwd(dy, saved, M, N, K, fmt, fmt_g, 0, wx, ww, bws,
                               *(got[n] if n in need else None for n in ("dx", "dw", "db")))
        for name in ("y", *need):
            gref.check_close(got[name], *want[name], f"{need} {name}")


def lut(fmt):
    return ref.decode(np.arange(256, dtype=np.uint8), fmt)


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("t,e,k,d,h", [
    (40, 64, 8, 1040, 528),     # no side a multiple of 128
    (160, 64, 8, 1040, 528),    # more than 16 tokens an expert
    (40, 64, 8, 1024, 512),
    (160, 64, 8, 1024, 512),
    (40, 64, 8, 1024, 528),
])
def test_experts(f, t, e, k, d, h, fmt):
    G = ref.groups
    rng = np.random.default_rng(t + d)
    x = wl.normal_bf16((t, d), 1.0, 1)
    r = wl.normal_bf16((e, d), 1.5 / np.sqrt(d), 2)
    w13, w2 = wl.random_codes((e, 2 * h, d), fmt, 3), wl.random_codes((e, d, h), fmt, 4)
    spread = 448 / 6 if fmt == 0 else 57344 / 16
    step = lambda n, *s: np.exp(rng.standard_normal(s) / 2).astype(np.float32) * np.float32(  # noqa: E731
        1 / spread / np.sqrt(n))
    s13, s2 = step(d, e, G(2 * h), G(d)), step(h, e, G(d), G(h))
    dev = lambda a: torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()  # noqa: E731
    out = torch.full((t * d + 64,), 0x7A11, dtype=torch.int16, device="cuda")
    ids = torch.empty(t, k, dtype=torch.int32, device="cuda")
    weights = torch.empty(t, k, device="cuda")
    ws = torch.zeros(f.fp8_moe_workspace(t, e, k, d, h), dtype=torch.uint8, device="cuda")
    args = [dev(a) for a in (x, r, w13, s13, w2, s2)]
    bits = []
    for _ in range(2):  # the second call finds the workspace as the first left it
        f.fp8_moe(*args, t, e, k, d, h, fmt, True, ws, out, ids=ids, weights=weights)
        torch.cuda.synchronize()
        bits.append(from_dev_bf16(out).copy())
    assert np.array_equal(*bits) and (bits[0][t * d:] == 0x7A11).all()
    ids, weights = ids.cpu().numpy(), weights.cpu().numpy()
    reached = len(np.unique(ids))
    assert -(-h // 32) * reached >= 1024 and -(-d // 64) * reached >= 1024
    v = lambda b: wl.bf16_bits_to_f32(b).astype(np.float64)  # noqa: E731
    table = lut(fmt)
    w13v = np.stack([table[w13[i]] * ref.grow(s13[i], 2 * h, d, 128, 128) for i in range(e)])
    w2v = np.stack([table[w2[i]] * ref.grow(s2[i], d, h, 128, 128) for i in range(e)])
    sample = np.unique(np.concatenate([[0, t - 1], rng.integers(0, t, 22)]))
    want, bound, wids, ww = ref.moe(v(x)[sample], v(r), w13v, w2v, k, True)
    np.testing.assert_array_equal(ids[sample], wids)
    np.testing.assert_allclose(weights[sample], ww, rtol=2e-5, atol=1e-30)
    ref.check_close(bits[0][:t * d].reshape(t, d)[sample], want, bound, f"{t} {d} {h}")
