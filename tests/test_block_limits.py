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
