"""Hidden activations of the expert layer at the end of the 32-bit range: one
unit's silu(gate) * up is beyond bf16's largest value, or beyond fp32's."""

import numpy as np
import pytest
import torch

import workloads as wl
from tests import block_ref as ref
from tests.gpu_util import from_dev_bf16

pytestmark = pytest.mark.gpu
D, H = 144, 48
ONE = (0x38, 0x3C)  # the code of 1


def run(t, fmt, gate_up, s2, dim=D, hidden=H):
    """One expert with weight 1: every token's hidden unit 3 is gate_up^2, its
    sign alternating by token, the others are 0; W2 is s2 times +1, -1 and 0 by
    turns for unit 3, and 0 for the others."""
    import fp8_tensor_scaled_amd as f
    one = ONE[fmt]
    x = np.zeros((t, dim), np.float32)
    x[:, 0] = np.where(np.arange(t) % 2, -1, 1)  # what the up row sees
    x[:, 1] = 1                                  # what the gate's sees
    w13 = np.zeros((2 * hidden, dim), np.uint8)
    w13[3, 1], w13[hidden + 3, 0] = one, one
    w2 = np.zeros((dim, hidden), np.uint8)
    w2[0::3, 3], w2[1::3, 3] = one, one | 0x80
    G = ref.groups
    s13 = np.full((G(2 * hidden), G(dim)), gate_up, np.float32)
    steps2 = np.full((G(dim), G(hidden)), s2, np.float32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    out = torch.empty(t, dim, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(f.fp8_moe_workspace(t, 1, 1, dim, hidden), dtype=torch.uint8, device="cuda")
    f.fp8_moe(dev(x).bfloat16(), torch.zeros(1, dim, dtype=torch.bfloat16, device="cuda"), dev(w13),
              dev(s13), dev(w2), dev(steps2), t, 1, 1, dim, hidden, fmt, True, ws, out)
    torch.cuda.synchronize()
    w13v = ref.decode(w13, fmt) * ref.grow(s13, 2 * hidden, dim, 128, 128)
    w2v = ref.decode(w2, fmt) * ref.grow(steps2, dim, hidden, 128, 128)
    return from_dev_bf16(out.view(torch.int16)), x.astype(float), w13v, w2v


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("t", [1, 2, 19])
def test_infinite_hidden_value(t, fmt):
    """1e20 * 1e20: infinite in 32 bits, and so are the outputs that take it
    with a weight other than 0 (infinity times 0 is NaN)."""
    got = wl.bf16_bits_to_f32(run(t, fmt, 1e20, 2.0 ** -10)[0])
    sign = np.where(np.arange(t) % 2, -1, 1)[:, None]
    assert np.array_equal(got[:, 0::3], np.broadcast_to(sign * np.inf, got[:, 0::3].shape))
    assert np.array_equal(got[:, 1::3], np.broadcast_to(-sign * np.inf, got[:, 1::3].shape))
    assert np.isnan(got[:, 2::3]).all()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("t", [1, 2, 19])
@pytest.mark.parametrize("square", [3.30e38, 3.393e38, 3.3965e38, 3.4e38])
def test_hidden_value_beyond_bf16(t, fmt, square):
    """Finite in 32 bits, some of them infinite when rounded to bf16: the
    outputs have the value, within the bound of 16 bits of precision."""
    got, x, w13, w2 = run(t, fmt, np.float32(np.sqrt(square)), 2.0 ** -100)
    out, bound, _, _ = ref.moe(x, np.zeros((1, x.shape[1])), w13[None], w2[None], 1, True)
    ref.check_close(got, out, bound, f"{t} {square}")
