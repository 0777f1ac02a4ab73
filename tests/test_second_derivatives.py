"""Second derivatives through the fp8 layers are refused (no GPU): the
gradients come from kernels, which autograd would take for constants."""

import ctypes

import pytest
import torch

from fp8_tensor_scaled_amd import autocast as ac

B16 = torch.bfloat16


@pytest.fixture(params=[ac.FP8Recipe(block=True), ac.FP8Recipe(dynamic=True)],
                ids=["block", "tensor"])
def layer(request, monkeypatch):
    for name in ("_linear_fwd_call", "_linear_block_fwd_call", "_on_gpu"):
        monkeypatch.setattr(ac, name, lambda *a: None)
    fill = lambda *outs: [t.fill_(2) for t in outs]  # noqa: E731
    monkeypatch.setattr(ac, "_linear_bwd_call", lambda *a: fill(*[t for t in a[13:15]
                                                                   if t is not None]))
    monkeypatch.setattr(ac, "_linear_block_bwd_call", lambda *a: fill(*[t for t in a[13:15]
                                                                         if t is not None]))
    monkeypatch.setattr(ac, "_stream", lambda s=None: ctypes.c_void_p(0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(ac, "_WS", {})

    def call(x, w):
        with ac.fp8_autocast(recipe=request.param):
            return ac.fp8_linear(x, w)
    return call


def test_refused(layer):
    x = torch.zeros(4, 48, dtype=B16, requires_grad=True)
    w = torch.zeros(32, 48, dtype=B16, requires_grad=True)
    y = layer(x, w)
    gx, = torch.autograd.grad(y, x, torch.zeros(4, 32, dtype=B16), create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated once"):
        (gx.square().sum() + w.sum()).backward(retain_graph=True)
    for leaf in (x, w):
        with pytest.raises(RuntimeError, match="differentiated once"):
            torch.autograd.grad(gx.square().sum() + leaf.sum(), leaf, retain_graph=True)
    # what does not go through the layer's gradient is not concerned
    v = torch.ones(3, requires_grad=True)
    gv, = torch.autograd.grad(gx.square().sum() + 3 * v.sum(), v)
    assert (gv == 3).all()


def test_output_gradient_with_a_history(layer):
    """dX depends on the output's gradient, which depends on v."""
    x = torch.zeros(4, 48, dtype=B16, requires_grad=True)
    w = torch.zeros(32, 48, dtype=B16)
    v = torch.ones(4, 32, dtype=B16, requires_grad=True)
    gx, = torch.autograd.grad((layer(x, w) * v).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated once"):
        torch.autograd.grad(gx.sum(), v)


def test_first_derivatives_as_without_a_graph(layer):
    x = torch.zeros(4, 48, dtype=B16, requires_grad=True)
    w = torch.zeros(32, 48, dtype=B16, requires_grad=True)
    y = layer(x, w)
    plain = torch.autograd.grad(y.sum(), [x, w], retain_graph=True)
    graphed = torch.autograd.grad(y.sum(), [x, w], create_graph=True)
    for a, b in zip(plain, graphed):
        assert torch.equal(a, b) and not a.requires_grad and b.requires_grad


def test_every_layer_is_marked():
    for fn in (ac._LinearFp8, ac._LinearFp8Weight, ac._LinearFp8Block):
        assert hasattr(fn.backward, "__wrapped__"), fn
