"""The block-scaled product split along k: shares of a tile in several
workgroups, added by the one that brings the last."""

import pytest
import torch

from tests import block_ref_gpu as ref

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1
COUNTERS = 1024  # bytes that a workspace begins with, zero between calls


@pytest.fixture(scope="module")
def f():
    import fp8_tensor_scaled_amd as f
    return f


def takes_the_short_kernel(layout, m, k):
    """Short A against a weight (rows of both along k), up to 64 groups: not split."""
    return layout == "nt" and m <= 64 and k <= 64 * ref.BLOCK


@pytest.mark.parametrize("layout,m,n,k,fa,fb,tile_b,bias", [
    ("nn", 128, 512, 4096, E5M2, E4M3, True, False),
    ("nn", 1000, 112, 4080, E4M3, E4M3, True, True),
    ("nn", 96, 208, 2560, E5M2, E5M2, False, True),
    ("tn", 256, 512, 4096, E5M2, E4M3, False, False),
    ("tn", 80, 160, 5003, E4M3, E4M3, False, True),     # k ends inside a group
    ("tn", 64, 64, 16384, E5M2, E5M2, True, False),
    ("nt", 100, 200, 4112, E4M3, E4M3, True, True),     # an uneven last share, odd output rows
    ("nt", 65, 333, 8208, E5M2, E4M3, True, False),
    ("nt", 130, 128, 6400, E5M2, E5M2, False, True),
    ("nt", 16, 128, 16384, E4M3, E4M3, True, False),    # few rows, long k
    ("nt", 1, 1, 32768, E4M3, E4M3, False, True),
])
def test_split_products(f, layout, m, n, k, fa, fb, tile_b, bias):
    need = f.fp8_mm_block_workspace(m, n, k)
    assert need > COUNTERS and not takes_the_short_kernel(layout, m, k)
    op = ref.Operands(layout, m, n, k, fa, fb, False, tile_b, bias, seed=m + n)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(3):
        outs.append(op.run(f, ws))
        assert not bool(ws[:COUNTERS].any()), "counters left"
    for out in outs[1:]:  # the shares are added in a fixed order
        assert ref.bits_equal(outs[0], out)
    op.check([outs[0], op.run(f)], f"{layout} {m}x{n}x{k}")


def test_one_workspace_for_many_shapes(f):
    shapes = [("nn", 128, 512, 4096), ("nt", 100, 200, 4112), ("tn", 256, 512, 4096)]
    ops = [ref.Operands(*s, E4M3, E4M3, False, s[0] != "tn", False, seed=i)
           for i, s in enumerate(shapes)]
    ws = torch.zeros(max(f.fp8_mm_block_workspace(*s[1:]) for s in shapes), dtype=torch.uint8,
                     device="cuda")
    for op in ops + ops[::-1]:
        op.check([op.run(f, ws)], str(op.shape))
