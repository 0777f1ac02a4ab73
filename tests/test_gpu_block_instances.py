"""Every kernel of the block-scaled product against the definition in 64 bits,
all outputs: each tile size in each layout, format and grouping, with ragged
sizes, and the layer's products made of them."""

import pytest
import torch

from tests import block_ref_gpu as ref

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1
FORMATS = [(E4M3, E4M3), (E5M2, E4M3), (E5M2, E5M2)]


@pytest.fixture(scope="module")
def f():
    import fp8_tensor_scaled_amd as f
    return f


def tile_cfg(m, n, bvec):
    """The rule by which a product of whole 16-byte rows gets its tile size."""
    tiles = lambda bm, bn: -(-m // bm) * -(-n // bn)        # noqa: E731
    rounds = lambda bm, bn: -(-tiles(bm, bn) // 256)        # noqa: E731
    if tiles(128, 128) < 128:
        return "small"
    wide = n >= m
    half = (rounds(128, 256) if wide else rounds(256, 128)) * (675 if bvec else 570)
    mid = rounds(128, 128) * (475 if bvec else 350)
    if not bvec and rounds(256, 256) * 1000 <= min(half, mid):
        return "big"
    return ("wide" if wide else "tall") if half <= mid else "mid"


SIZES = {"big": (4080, 4080), "wide": (2032, 4080), "tall": (4080, 2032), "mid": (2032, 2032),
         "small": (1008, 944)}


# (there is no 256 x 256 kernel with a step per column of B)
TILES = [(cfg, tile_b) for cfg in SIZES for tile_b in (True, False) if tile_b or cfg != "big"]


@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("cfg,tile_b", TILES)
@pytest.mark.parametrize("layout", ["nt", "nn", "tn"])
def test_tiles(f, layout, cfg, tile_b, fa, fb):
    m, n = SIZES[cfg]
    m += layout != "tn"                 # (rows of A that are no multiple of 16 where
    k = 527 if layout == "tn" else 528  # the layout allows it; k ends inside a group)
    assert tile_cfg(m, n, not tile_b) == cfg
    op = ref.Operands(layout, m, n, k, fa, fb, False, tile_b, fa == fb, seed=m + fa)
    op.check([op.run(f)], f"{layout} {cfg}")


@pytest.mark.parametrize("cfg,tile_b", TILES)
def test_tiles_with_odd_output_rows(f, cfg, tile_b):
    m, n = SIZES[cfg]
    n -= 3
    assert tile_cfg(m, n, not tile_b) == cfg
    op = ref.Operands("nt", m, n, 272, E4M3, E4M3, False, tile_b, True, seed=m)
    op.check([op.run(f)], cfg)


@pytest.mark.parametrize("cfg", list(SIZES))
@pytest.mark.parametrize("layout", ["nt", "nn", "tn"])
@pytest.mark.parametrize("k", [16, 128, 384, 1040])
def test_tiles_short_and_long(f, layout, cfg, k):
    """One group, whole ones, more stages than the ring has; a step per tile of A too."""
    m, n = SIZES[cfg]
    op = ref.Operands(layout, m, n, k, E5M2, E4M3, True, True, False, seed=k)
    op.check([op.run(f)], f"{layout} {cfg} {k}")


@pytest.mark.parametrize("fa,fb", FORMATS + [(E4M3, E5M2)])
@pytest.mark.parametrize("layout", ["nt", "nn", "tn", "tt"])
def test_any_alignment_large(f, layout, fa, fb):
    """The general kernel's 128 x 128 tiles: from 256 of them on, rows that
    begin anywhere, every side ragged."""
    m, n, k = 2047, 2049, 531
    op = ref.Operands(layout, m, n, k, fa, fb, False, layout != "tn", True, seed=fa + 2 * fb)
    op.check([op.run(f)], layout)


@pytest.mark.parametrize("layout", ["nt", "nn", "tn"])
@pytest.mark.parametrize("k", [16, 17, 127, 129, 1027])
def test_any_alignment_depths(f, layout, k):
    op = ref.Operands(layout, 2050, 2011, k, E4M3, E4M3, True, False, False, seed=k)
    op.check([op.run(f)], f"{layout} {k}")


@pytest.mark.parametrize("M,N,K", [(1000, 1040, 1072), (2048, 2816, 2064), (4096, 4096, 528),
                                   (1001, 1043, 1070)])
@pytest.mark.parametrize("fmt,fmt_g", [(E4M3, E5M2), (E4M3, E4M3), (E5M2, E5M2)])
def test_layer(f, M, N, K, fmt, fmt_g):
    """Output and gradients of the layer from its operands' codes (those of
    fp8_quantize_block): both gradients in one launch, each in its own, sides
    that the tiled kernels do not take."""
    r = lambda *s, seed: torch.randn(*s, device="cuda",  # noqa: E731
                                     generator=ref.generator(seed)).bfloat16()
    x, w, dy, bias = r(M, K, seed=1), r(N, K, seed=2), r(M, N, seed=3), r(N, seed=4)
    buf = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    b16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    saved = buf(f.fp8_linear_block_saved(M, N, K, True, True))
    y, dx, dw, db = b16(M, N), b16(M, K), b16(N, K), b16(N)
    f.fp8_linear_block_fwd(x, w, bias, M, N, K, fmt, 0, saved, True, True,
                           buf(f.fp8_linear_block_fwd_workspace(M, N, K)), y)
    f.fp8_linear_block_bwd(dy, saved, M, N, K, fmt, fmt_g, 0, True, True,
                           buf(f.fp8_linear_block_bwd_workspace(M, N, K)), dx, dw, db)

    def quantize(t, rows, cols, ft, kind):
        c = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        s = torch.empty({"row": (rows, ref.groups(cols)), "col": (ref.groups(rows), cols),
                         "tile": (ref.groups(rows), ref.groups(cols))}[kind], device="cuda")
        f.fp8_quantize_block(t, rows, cols, ft, **{"out_" + kind: c, "scale_" + kind: s})
        return ref.decode(c, ft), s

    wq, sw = quantize(w, N, K, fmt, "tile")
    xr, sxr = quantize(x, M, K, fmt, "row")
    ref.check_close(y, *ref.product(xr, wq.t(), sxr, sw.repeat_interleave(128, 0)[:N].t(), bias),
                    "y")
    gr, sgr = quantize(dy, M, N, fmt_g, "row")
    ref.check_close(dx, *ref.product(gr, wq, sgr, sw.repeat_interleave(128, 1)[:, :K]), "dx")
    gc, sgc = quantize(dy, M, N, fmt_g, "col")
    xc, sxc = quantize(x, M, K, fmt, "col")
    ref.check_close(dw, *ref.product(gc.t(), xc, sgc.t(), sxc), "dw")
    ref.check_close(db, dy.double().sum(0), M * 2.0 ** -24 * dy.double().abs().sum(0), "db")
