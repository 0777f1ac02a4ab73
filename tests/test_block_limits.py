"""Limits of the block-scaled entry points beyond those of their first tests
(no GPU): row strides, alignment of every operand."""

import ctypes

import pytest

import fp8_tensor_scaled_amd as f

P = ctypes.c_void_p
FAKE = P(0x1000)  # never dereferenced: validation fails first


def err():
    return f._lib.fp8_last_error().decode()


def layer_args(M, N, K, backward, **over):
    """Arguments of fp8_linear_block_fwd / _bwd, right but for `over`."""
    saved = f.fp8_linear_block_saved(M, N, K, True, True)
    if backward:
        a = dict(g=FAKE, saved=FAKE, saved_bytes=saved, w8=None, sw=None, fmt_w=0, M=M, N=N, K=K,
                 fmt=0, fmt_g=1, margin=0, want_dx=1, want_dw=1, workspace=FAKE,
                 workspace_bytes=f.fp8_linear_block_bwd_workspace(M, N, K), dx=FAKE, dw=FAKE,
                 db=FAKE, stream=None)
    else:
        a = dict(x=FAKE, w=FAKE, w8=None, sw=None, fmt_w=0, bias=FAKE, M=M, N=N, K=K, fmt=0,
                 margin=0, saved=FAKE, saved_bytes=saved, want_dx=1, want_dw=1, workspace=FAKE,
                 workspace_bytes=f.fp8_linear_block_fwd_workspace(M, N, K), out=FAKE, stream=None)
    a.update(over)
    return list(a.values())


def call(backward):
    return f._lib.fp8_linear_block_bwd if backward else f._lib.fp8_linear_block_fwd


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("M,N,K", [(4, 8, 1 << 24), (4, 1 << 24, 8), (1, 128, 33900001),
                                   (1, 33900001, 128)])
def test_layer_row_strides(backward, M, N, K):
    """N and K are the operands' row strides in the products, whose general
    kernel reaches a tile's rows (up to 127 of them) by 32-bit offsets: as
    fp8_mm_block, below 2^24."""
    assert call(backward)(*layer_args(M, N, K, backward)) == 1 and "below 2^24" in err(), err()


ODD, HALF = P(0x1001), P(0x1002)  # not aligned to bf16, to fp32


@pytest.mark.parametrize("backward,over", [
    (False, dict(x=ODD)), (False, dict(w=ODD)), (False, dict(bias=ODD)), (False, dict(out=ODD)),
    (False, dict(w=None, w8=FAKE, sw=HALF)), (True, dict(g=ODD)), (True, dict(dx=ODD)),
    (True, dict(dw=ODD)), (True, dict(db=ODD)), (True, dict(w8=FAKE, sw=HALF))])
def test_layer_alignment(backward, over):
    """The steps of a weight's tiles are loaded into LDS by whole dwords."""
    args = layer_args(4, 200, 300, backward, **over)
    assert call(backward)(*args) == 1 and "aligned to its elements" in err(), err()


@pytest.mark.parametrize("steps", ["scale_row", "scale_col", "scale_tile"])
def test_quantize_alignment(steps):
    a = dict(x=FAKE, in_type=0, rows=4, cols=200, ldx=200, fmt=0, margin=0, out_row=None,
             scale_row=None, out_col=None, scale_col=None, out_tile=None, scale_tile=None,
             stream=None)
    a.update({steps: HALF, steps.replace("scale", "out"): FAKE})
    assert f._lib.fp8_quantize_block(*a.values()) == 1 and "aligned to its elements" in err(), err()
