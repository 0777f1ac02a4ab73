"""Block quantize of matrices with more tiles than one grid dimension of the
runtime holds (2^32 lanes): the codes and steps of quantizing them in parts.
Values repeat every `PERIOD`, so that a small call gives what is expected."""

import pytest
import torch

pytestmark = pytest.mark.gpu
PERIOD = 128 * 999


@pytest.fixture(scope="module")
def long():
    n = (1 << 31) + 128 * 5 + 37
    g = torch.Generator(device="cuda").manual_seed(1)
    part = torch.randn(PERIOD, device="cuda", generator=g).bfloat16()
    return n, part, part.repeat(-(-n // PERIOD))[:n]


def check(whole, part):
    """whole is part, over and over."""
    n, p = whole.numel(), part.numel()
    full = n // p * p
    w = whole.reshape(-1)
    assert bool((w[:full].view(-1, p) == part.reshape(-1)).all())
    assert torch.equal(w[full:], part.reshape(-1)[:n - full])


@pytest.mark.parametrize("kind", ["row", "tile"])
def test_one_long_row(long, kind):
    import fp8_tensor_scaled_amd as f
    n, part, x = long

    def quantize(v):
        m = v.numel()
        codes = torch.empty(m, dtype=torch.uint8, device="cuda")
        steps = torch.empty((m + 127) // 128, device="cuda")
        f.fp8_quantize_block(v, 1, m, f.E4M3, **{"out_" + kind: codes, "scale_" + kind: steps})
        return codes, steps

    codes, steps = quantize(x)
    want, want_steps = quantize(part)
    tail = n // 128 * 128  # the last group is a part of one
    check(codes[:tail], want)
    check(steps[:-1], want_steps)
    last, last_step = quantize(x[tail:].clone())
    assert torch.equal(codes[tail:], last) and torch.equal(steps[-1:], last_step)


def test_one_long_column(long):
    import fp8_tensor_scaled_amd as f
    n, part, x = long

    def quantize(v):
        m = v.numel()
        codes = torch.empty(m, dtype=torch.uint8, device="cuda")
        steps = torch.empty((m + 127) // 128, device="cuda")
        f.fp8_quantize_block(v, m, 1, f.E4M3, out_col=codes, scale_col=steps)
        return codes, steps

    codes, steps = quantize(x)
    want, want_steps = quantize(part)
    tail = n // 128 * 128
    check(codes[:tail], want)
    check(steps[:-1], want_steps)
    last, last_step = quantize(x[tail:].clone())
    assert torch.equal(codes[tail:], last) and torch.equal(steps[-1:], last_step)
