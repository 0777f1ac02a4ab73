"""Host checks of the block-scaled entry points (no GPU): every refusal of
the C functions and of their Python binding, and the recipe's checks."""

import ctypes

import pytest
import torch

import fp8_tensor_scaled_amd as f
from fp8_tensor_scaled_amd import autocast as ac

P = ctypes.c_void_p
FAKE, FAKE2 = P(0x1000), P(0x80000)  # never dereferenced: validation fails first


def err():
    return f._lib.fp8_last_error().decode()


def quantize_args(**over):
    a = dict(x=FAKE, in_type=0, rows=4, cols=200, ldx=200, fmt=0, margin=0, out_row=FAKE,
             scale_row=FAKE, out_col=None, scale_col=None, out_tile=None, scale_tile=None,
             stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,needle", [
    (dict(fmt=2), "format"),
    (dict(in_type=3), "input type"),
    (dict(rows=-1), ">= 0"),
    (dict(cols=-1), ">= 0"),
    (dict(ldx=199), "ldx 199 < cols 200"),
    (dict(margin=65), "margin"),
    (dict(margin=-1), "margin"),
    (dict(scale_row=None), "go together"),
    (dict(out_row=None), "go together"),
    (dict(out_col=FAKE2), "go together"),
    (dict(scale_tile=FAKE2), "go together"),
    (dict(out_row=None, scale_row=None), "no output"),
    (dict(out_tile=FAKE2, scale_tile=FAKE2), "tiles go alone"),
    (dict(x=None), "x is NULL"),
    (dict(x=P(0x1001)), "aligned"),
    (dict(x=P(0x1002), in_type=2), "aligned"),
    (dict(out_col=P(0x1000 + 799), scale_col=FAKE2), "overlap"),
    (dict(rows=1 << 30, cols=1 << 20, ldx=1 << 20), "too many blocks"),
    (dict(rows=1 << 40, cols=1 << 20, ldx=1 << 20), "too many elements"),
])
def test_quantize_block_refusals(over, needle):
    assert f._lib.fp8_quantize_block(*quantize_args(**over)) == 1 and needle in err(), err()


def test_quantize_block_empty_does_nothing():
    assert f._lib.fp8_quantize_block(*quantize_args(rows=0, x=None)) == 0
    assert f._lib.fp8_quantize_block(*quantize_args(cols=0, ldx=0, x=None)) == 0


def mm_args(**over):
    a = dict(a=FAKE, b=FAKE, fmt_a=0, fmt_b=0, trans_a=0, trans_b=1, m=4, n=8, k=300, lda=300,
             ldb=300, scale_a=FAKE, group_a=0, scale_b=FAKE, group_b=1, bias=None, out=FAKE,
             workspace=None, workspace_bytes=0, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,needle", [
    (dict(fmt_a=2), "format"),
    (dict(fmt_b=-1), "format"),
    (dict(a=None), "NULL"),
    (dict(b=None), "NULL"),
    (dict(out=None), "NULL"),
    (dict(scale_a=None), "NULL"),
    (dict(scale_b=None), "NULL"),
    (dict(trans_a=2), "trans"),
    (dict(trans_b=-1), "trans"),
    (dict(group_a=2), "grouping"),
    (dict(group_b=-1), "grouping"),
    (dict(m=0), ">= 1"),
    (dict(n=0), ">= 1"),
    (dict(k=0), ">= 1"),
    (dict(lda=299), "lda 299 < 300"),
    (dict(ldb=299), "ldb 299 < 300"),
    (dict(trans_a=1, lda=3), "lda 3 < 4"),
    (dict(trans_b=0, ldb=7), "ldb 7 < 8"),
    (dict(m=1 << 30, n=1 << 20), "too large"),
    (dict(m=1 << 39, n=1, lda=1 << 23), "too large"),
    (dict(lda=1 << 24), "below 2^24"),
    (dict(ldb=1 << 24), "below 2^24"),
    (dict(out=P(0x1001)), "aligned"),
    (dict(bias=P(0x1001)), "aligned"),
    (dict(scale_a=P(0x1002)), "aligned"),
    (dict(workspace=P(0x1010), workspace_bytes=1 << 30), "256-byte"),
])
def test_mm_block_refusals(over, needle):
    assert f._lib.fp8_mm_block(*mm_args(**over)) == 1 and needle in err(), err()


def test_mm_block_workspace_sizes():
    assert f.fp8_mm_block_workspace(0, 1, 1) == 0
    for m, n, k in ((1, 128, 8192), (16, 1024, 4096), (4096, 4096, 4096), (64, 512, 65536)):
        need = f.fp8_mm_block_workspace(m, n, k)
        if need:
            args = mm_args(m=m, n=n, k=k, lda=k, ldb=k, workspace=FAKE, workspace_bytes=need - 1)
            assert f._lib.fp8_mm_block(*args) == 1 and "workspace" in err()


def fwd_args(**over):
    need = f.fp8_linear_block_saved(4, 200, 300, True, True)
    a = dict(x=FAKE, w=FAKE, w8=None, sw=None, fmt_w=0, bias=None, M=4, N=200, K=300, fmt=0,
             margin=0, saved=FAKE, saved_bytes=need, want_dx=1, want_dw=1, workspace=FAKE,
             workspace_bytes=f.fp8_linear_block_fwd_workspace(4, 200, 300), out=FAKE, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,needle", [
    (dict(fmt=2), "format"),
    (dict(w=None, w8=FAKE, sw=FAKE, fmt_w=5), "format"),
    (dict(x=None), "NULL"),
    (dict(out=None), "NULL"),
    (dict(w=None), "either as bf16 or as codes"),
    (dict(w8=FAKE, sw=FAKE), "either as bf16 or as codes"),
    (dict(w=None, w8=FAKE), "need their steps"),
    (dict(M=0), ">= 1"),
    (dict(M=1 << 30, K=1 << 20), "too large"),
    (dict(margin=65), "margin"),
    (dict(saved=None), "saved is NULL"),
    (dict(saved_bytes=100), "saved 100 <"),
    (dict(saved=P(0x1010)), "256-byte"),
    (dict(workspace=None), "workspace is NULL"),
    (dict(workspace_bytes=6656), "workspace 6656 <"),
    (dict(workspace=P(0x1010)), "256-byte"),
])
def test_linear_block_fwd_refusals(over, needle):
    assert f._lib.fp8_linear_block_fwd(*fwd_args(**over)) == 1 and needle in err(), err()


def bwd_args(**over):
    need = f.fp8_linear_block_saved(4, 200, 300, True, True)
    a = dict(g=FAKE, saved=FAKE, saved_bytes=need, w8=None, sw=None, fmt_w=0, M=4, N=200, K=300,
             fmt=0, fmt_g=1, margin=0, want_dx=1, want_dw=1, workspace=FAKE,
             workspace_bytes=f.fp8_linear_block_bwd_workspace(4, 200, 300), dx=FAKE, dw=FAKE,
             db=None, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,needle", [
    (dict(fmt=2), "format"),
    (dict(fmt_g=2), "format"),
    (dict(g=None), "g is NULL"),
    (dict(w8=FAKE), "need their steps"),
    (dict(K=0), ">= 1"),
    (dict(margin=-1), "margin"),
    (dict(want_dx=0), "did not keep"),
    (dict(want_dw=0), "did not keep"),
    (dict(saved=None), "saved is NULL"),
    (dict(saved_bytes=100), "saved 100 <"),
    (dict(workspace_bytes=7000), "workspace 7000 <"),
])
def test_linear_block_bwd_refusals(over, needle):
    assert f._lib.fp8_linear_block_bwd(*bwd_args(**over)) == 1 and needle in err(), err()


def test_linear_block_buffers():
    """The binding's own checks: sizes, types, and that tensors are on a GPU."""
    fwd = dict(x=b16(1200), w=b16(60000), bias=None, M=4, N=200, K=300, fmt=0, margin=0,
               saved=None, want_dx=False, want_dw=False, workspace=u8(1 << 20), out=b16(800))
    raises("x: 1199 elements", lambda: f.fp8_linear_block_fwd(**dict(fwd, x=b16(1199))))
    raises("w: 59999 elements", lambda: f.fp8_linear_block_fwd(**dict(fwd, w=b16(59999))))
    raises("out: 799 elements", lambda: f.fp8_linear_block_fwd(**dict(fwd, out=b16(799))))
    raises("bias: 199 elements", lambda: f.fp8_linear_block_fwd(**dict(fwd, bias=b16(199))))
    raises("sw: 5 elements", lambda: f.fp8_linear_block_fwd(**dict(fwd, w=None, w8=u8(60000),
                                                                   sw=f32(5))))
    raises("is on cpu, not a GPU", lambda: f.fp8_linear_block_fwd(**fwd))
    raises("negative size", lambda: f.fp8_linear_block_fwd(**dict(fwd, M=-1)))
    bwd = dict(g=b16(800), saved=None, M=4, N=200, K=300, fmt=0, fmt_g=1, margin=0, want_dx=False,
               want_dw=False, workspace=u8(1 << 20), dx=b16(1200), dw=b16(60000), db=b16(200))
    for name, n in (("g", 800), ("dx", 1200), ("dw", 60000), ("db", 200)):
        raises(f"{name}: {n - 1} elements",
               lambda: f.fp8_linear_block_bwd(**dict(bwd, **{name: b16(n - 1)})))
    raises("is on cpu, not a GPU", lambda: f.fp8_linear_block_bwd(**bwd))


def test_linear_block_sizes():
    assert f.fp8_linear_block_saved(0, 1, 1, True, True) == 0
    assert f.fp8_linear_block_saved(4, 200, 300, False, False) == 0
    both = f.fp8_linear_block_saved(4, 200, 300, True, True)
    assert both >= 4 * 300 + 4 * 300 + 200 * 300 + 4 * 2 * 3
    assert f.fp8_linear_block_saved(4, 200, 300, True, False) < both
    assert f.fp8_linear_block_fwd_workspace(4, 200, 300) > 6656 + 4 * 300 + 200 * 300


def moe_args(**over):
    a = dict(x=FAKE, router=FAKE, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, tokens=4, experts=8,
             top_k=2, dim=256, hidden=128, fmt=0, renormalize=1, workspace=FAKE,
             workspace_bytes=1 << 40, out=FAKE, ids=None, weights=None, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,needle", [
    (dict(fmt=3), "format"),
    (dict(tokens=-1), "tokens"),
    (dict(tokens=1025), "tokens"),
    (dict(experts=0), "experts"),
    (dict(experts=513), "experts"),
    (dict(top_k=0), "top_k"),
    (dict(top_k=9), "top_k"),
    (dict(experts=64, top_k=17), "top_k"),
    (dict(dim=8), "dim"),
    (dict(dim=264), "dim"),
    (dict(hidden=0), "hidden"),
    (dict(hidden=100), "hidden"),
    (dict(x=None), "NULL"),
    (dict(router=None), "NULL"),
    (dict(w13=None), "NULL"),
    (dict(s13=None), "NULL"),
    (dict(w2=None), "NULL"),
    (dict(s2=None), "NULL"),
    (dict(workspace=None), "NULL"),
    (dict(out=None), "NULL"),
    (dict(x=P(0x1002)), "16-byte"),
    (dict(w2=P(0x1008)), "16-byte"),
    (dict(s2=P(0x1002)), "aligned"),
    (dict(ids=P(0x1002)), "aligned"),
    (dict(workspace_bytes=0), "workspace"),
    (dict(workspace=P(0x1010)), "256-byte"),
])
def test_moe_refusals(over, needle):
    assert f._lib.fp8_moe(*moe_args(**over)) == 1 and needle in err(), err()


def test_moe_without_tokens_does_nothing():
    assert f._lib.fp8_moe(*moe_args(tokens=0, x=None, out=None, workspace_bytes=0)) == 0
    assert f.fp8_moe_workspace(4, 8, 9, 256, 128) == 0
    assert f.fp8_moe_workspace(4, 8, 2, 256, 128) > 0


# ---- the binding: buffers against the sizes the C side will assume --------

u8 = lambda n: torch.empty(n, dtype=torch.uint8)      # noqa: E731
b16 = lambda n: torch.empty(n, dtype=torch.bfloat16)  # noqa: E731
f32 = lambda n: torch.empty(n, dtype=torch.float32)   # noqa: E731


def raises(needle, fn, *a, **kw):
    with pytest.raises(ValueError, match=needle):
        fn(*a, **kw)


def test_quantize_block_buffers():
    q, x = f.fp8_quantize_block, b16(3 * 200)
    raises("x: 600 elements, needs at least 800", q, x, 4, 200, f.E4M3, u8(800), f32(8))
    raises("x: 600 elements, needs at least 602", q, x, 3, 200, f.E4M3, u8(600), f32(6), ldx=201)
    raises("out_row: 599 elements", q, x, 3, 200, f.E4M3, u8(599), f32(6))
    raises("scale_row: 5 elements, needs at least 6", q, x, 3, 200, f.E4M3, u8(600), f32(5))
    raises("scale_row: required", q, x, 3, 200, f.E4M3, u8(600))
    raises("scale_col: 199 elements", q, x, 3, 200, f.E4M3, out_col=u8(600), scale_col=f32(199))
    raises("scale_tile: 1 elements", q, x, 3, 200, f.E4M3, out_tile=u8(600), scale_tile=f32(1))
    raises("out_tile: dtype", q, x, 3, 200, f.E4M3, out_tile=b16(600), scale_tile=f32(2))
    raises("bad sizes", q, x, 3, 200, f.E4M3, u8(600), f32(6), ldx=199)
    raises("no input type", q, f32(600).double(), 3, 200, f.E4M3, u8(600), f32(6))
    raises("for input type", q, x, 3, 200, f.E4M3, u8(600), f32(6), in_type=f.IN_F32)
    raises("bad input type", q, x, 3, 200, f.E4M3, u8(600), f32(6), in_type=7)
    raises("must be contiguous", q, b16(1200)[::2], 3, 200, f.E4M3, u8(600), f32(6))
    raises("must be contiguous", q, b16(900).view(3, 300)[:, :200], 3, 200, f.E4M3, u8(600),
           f32(6))
    # a slice of a wider tensor's columns, with its row stride
    raises("is on cpu, not a GPU", q, b16(900).view(3, 300)[:, :200], 3, 200, f.E4M3, u8(600),
           f32(6), ldx=300)


def mm(**over):
    """An NT 3 x 5 x 300 product with row steps for A and tile steps for B."""
    a = dict(a=u8(900), b=u8(1500), fmt_a=f.E4M3, fmt_b=f.E4M3, trans_a=0, trans_b=1, m=3, n=5,
             k=300, lda=300, ldb=300, scale_a=f32(9), group_a=f.GROUP_LINE, scale_b=f32(3),
             group_b=f.GROUP_TILE, bias=None, out=b16(15))
    a.update(over)
    return a


def test_mm_block_buffers():
    raises("a: 899 elements", lambda: f.fp8_mm_block(**mm(a=u8(899))))
    raises("b: 1499 elements", lambda: f.fp8_mm_block(**mm(b=u8(1499))))
    raises("b: 1500 elements, needs at least 1504", lambda: f.fp8_mm_block(**mm(ldb=301)))
    raises("scale_a: 8 elements, needs at least 9", lambda: f.fp8_mm_block(**mm(scale_a=f32(8))))
    raises("scale_b: 2 elements, needs at least 3", lambda: f.fp8_mm_block(**mm(scale_b=f32(2))))
    raises("scale_b: 3 elements, needs at least 15",
           lambda: f.fp8_mm_block(**mm(group_b=f.GROUP_LINE)))
    raises("bias: 4 elements", lambda: f.fp8_mm_block(**mm(bias=b16(4))))
    raises("out: 14 elements", lambda: f.fp8_mm_block(**mm(out=b16(14))))
    raises("out: dtype torch.float16", lambda: f.fp8_mm_block(**mm(out=b16(15).half())))
    raises("bad grouping", lambda: f.fp8_mm_block(**mm(group_a=3)))
    raises("negative size", lambda: f.fp8_mm_block(**mm(m=-1)))
    raises("is on cpu, not a GPU", lambda: f.fp8_mm_block(**mm()))


def moe(**over):
    a = dict(x=b16(512), router=b16(4 * 256), w13=u8(4 * 256 * 256), s13=f32(16),
             w2=u8(4 * 256 * 128), s2=f32(8), tokens=2, experts=4, top_k=2, dim=256, hidden=128,
             fmt=f.E4M3, renormalize=True, workspace=u8(1 << 16), out=b16(512))
    a.update(over)
    return a


def test_moe_buffers():
    raises("x: 511 elements", lambda: f.fp8_moe(**moe(x=b16(511))))
    raises("x: dtype torch.float16", lambda: f.fp8_moe(**moe(x=b16(512).half())))
    raises("router: 1023 elements", lambda: f.fp8_moe(**moe(router=b16(1023))))
    raises("w13: 262143 elements", lambda: f.fp8_moe(**moe(w13=u8(4 * 256 * 256 - 1))))
    raises("s13: 15 elements", lambda: f.fp8_moe(**moe(s13=f32(15))))
    raises("w2: 131071 elements", lambda: f.fp8_moe(**moe(w2=u8(4 * 256 * 128 - 1))))
    raises("s2: 7 elements", lambda: f.fp8_moe(**moe(s2=f32(7))))
    raises("out: 511 elements", lambda: f.fp8_moe(**moe(out=b16(511))))
    raises("ids: dtype torch.int64", lambda: f.fp8_moe(**moe(ids=torch.empty(4, dtype=torch.int64))))
    raises("weights: 3 elements", lambda: f.fp8_moe(**moe(weights=f32(3))))
    raises("negative size", lambda: f.fp8_moe(**moe(tokens=-1)))
    raises("is on cpu, not a GPU", lambda: f.fp8_moe(**moe()))


# ---- the recipe -----------------------------------------------------------

def test_block_recipe():
    assert not ac.FP8Recipe().block
    assert ac.FP8Recipe(block=True, margin=2).margin == 2
    with pytest.raises(ValueError, match="dynamic does not apply"):
        ac.FP8Recipe(block=True, dynamic=True)
    with ac.fp8_autocast(recipe=ac.FP8Recipe(block=True)):
        w8 = torch.zeros(256, 300, dtype=torch.uint8).view(torch.float8_e4m3fn)
        x = torch.zeros(2, 300, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="a step for each 128 x 128 tile"):
            ac.fp8_linear(x, w8, w_scale=torch.ones(1))
        with pytest.raises(ValueError, match="must be float32"):
            ac.fp8_linear(x, w8, w_scale=torch.ones(2, 3, dtype=torch.float64))
        with pytest.raises(ValueError, match="on one GPU"):
            ac.fp8_linear(x, w8, w_scale=torch.ones(2, 3))
        with pytest.raises(ValueError, match="on one GPU"):
            ac.fp8_linear(x, torch.zeros(256, 300, dtype=torch.bfloat16))
        with pytest.raises(ValueError, match="bf16 bias"):
            ac.fp8_linear(x, w8, w_scale=torch.ones(2, 3), b_scale=torch.ones(1),
                          bias=torch.zeros(256, dtype=torch.uint8).view(torch.float8_e4m3fn))


def test_expert_module_refuses_host_tensors():
    from fp8_tensor_scaled_amd.moe import FP8MoE
    b16 = torch.bfloat16
    with pytest.raises(ValueError, match="router must be a 2-D bfloat16 tensor on the GPU"):
        FP8MoE(torch.zeros(4, 64, dtype=b16), torch.zeros(4, 64, 64, dtype=b16),
               torch.zeros(4, 64, 32, dtype=b16), 2)
