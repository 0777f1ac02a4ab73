"""Inputs of the expert module that begin anywhere, and its state after a
model's conversions."""

import pytest
import torch

from fp8_tensor_scaled_amd.moe import FP8MoE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def module():
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: (torch.randn(*s, device="cuda", generator=g) * 0.1).bfloat16()  # noqa: E731
    return FP8MoE(r(6, 144), r(6, 160, 144), r(6, 144, 80), 2)


@pytest.mark.parametrize("off", [1, 3, 4, 8])
@pytest.mark.parametrize("tokens", [1, 13])
def test_any_alignment(module, off, tokens):
    """A contiguous view whose first element lies `off` elements into a buffer."""
    flat = torch.randn(off + tokens * 144, device="cuda").bfloat16()
    x = flat[off:].view(tokens, 144)
    assert x.is_contiguous() and x.data_ptr() % 16 == 2 * off % 16
    assert torch.equal(module(x), module(x.clone()))
    assert torch.equal(module(x[0]), module(x[:1].clone())[0])


def test_after_a_conversion(module):
    x = torch.randn(5, 144, device="cuda").bfloat16()
    y = module(x)
    for convert in (lambda m: m.half(), lambda m: m.float(), lambda m: m.to(torch.bfloat16)):
        assert torch.equal(convert(torch.nn.Sequential(module))[0](x), y)
