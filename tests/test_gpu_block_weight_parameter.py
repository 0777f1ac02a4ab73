"""A weight of codes kept as a Parameter (torch's default: it requires a
gradient) takes none, and nothing is kept for one."""

import pytest
import torch

from fp8_tensor_scaled_amd.autocast import FP8Recipe, fp8_autocast, fp8_linear

pytestmark = pytest.mark.gpu


def test_codes_as_a_parameter():
    import fp8_tensor_scaled_amd as f
    w = torch.randn(144, 272, device="cuda").bfloat16()
    w8 = torch.empty(144, 272, dtype=torch.float8_e4m3fn, device="cuda")
    sw = torch.empty(2, 3, device="cuda")
    f.fp8_quantize_block(w, 144, 272, f.E4M3, out_tile=w8, scale_tile=sw)
    g = torch.randn(20, 144, device="cuda").bfloat16()
    x0 = torch.randn(20, 272, device="cuda").bfloat16()
    grads = []
    for weight in (w8, torch.nn.Parameter(w8)):
        x = x0.clone().requires_grad_()
        with fp8_autocast(recipe=FP8Recipe(block=True)):
            y = fp8_linear(x, weight, w_scale=sw)
        kept = [t for t in y.grad_fn.saved_tensors if t is not None]
        assert {t.data_ptr() for t in kept} == {w8.data_ptr(), sw.data_ptr()}
        y.backward(g)
        assert weight.grad is None
        grads.append(x.grad)
    assert torch.equal(*grads)
