"""FP8MoE's buffers (no GPU): what a conversion of the whole model leaves."""

import copy

import pytest
import torch

from fp8_tensor_scaled_amd.moe import FP8MoE

B16 = torch.bfloat16


def module():
    m = FP8MoE.__new__(FP8MoE)
    torch.nn.Module.__init__(m)
    m.top_k, m.renormalize, m.fmt = 2, True, 0
    g = torch.Generator().manual_seed(1)
    m.register_buffer("router", torch.randn(4, 64, generator=g).to(B16))
    m.register_buffer("w13", torch.randint(0, 255, (4, 64, 64), dtype=torch.uint8, generator=g))
    m.register_buffer("w13_steps", torch.rand(4, 1, 1, generator=g))
    m.register_buffer("w2", torch.randint(0, 255, (4, 64, 32), dtype=torch.uint8, generator=g))
    m.register_buffer("w2_steps", torch.rand(4, 1, 1, generator=g))
    return m


@pytest.mark.parametrize("convert", [lambda m: m.to(B16), lambda m: m.half(), lambda m: m.float(),
                                     lambda m: m.double(), lambda m: m.to(torch.float16).float(),
                                     lambda m: copy.deepcopy(m).bfloat16()])
def test_conversions_leave_types_and_values(convert):
    m, want = module(), module().state_dict()
    model = convert(torch.nn.Sequential(torch.nn.Linear(2, 2), m))
    got = model[1].state_dict()
    assert list(got) == list(want)
    for name, t in want.items():
        assert got[name].dtype == t.dtype and torch.equal(got[name], t), name


def test_moves_still_move():
    m = module().to("meta")
    assert all(t.device.type == "meta" for t in m.state_dict().values())
    assert m.router.dtype == B16 and m.w2_steps.dtype == torch.float32
    assert m.to_empty(device="cpu").w13_steps.device.type == "cpu"
