"""Workspaces of captured layer calls (no GPU): a graph's scratch is its own.
A buffer kept for eager calls would be cleared by the graph's replays only, or
replaced by a larger one while replays still write to it."""

import ctypes

import pytest
import torch

from fp8_tensor_scaled_amd import autocast as ac

B16 = torch.bfloat16
CONTROL = 6656  # bytes that begin a tensor-scaled call's workspace, zero between calls


@pytest.fixture
def handed(monkeypatch):
    """Workspaces handed to stand-in library calls, which leave them dirty."""
    got = []

    def call(*args, **kw):
        ws = next(a for a in args if isinstance(a, torch.Tensor) and a.dtype == torch.uint8)
        got.append((ws, ws[:CONTROL].clone()))
        ws.fill_(0xAB)

    for name in ("_linear_fwd_call", "_linear_bwd_call"):
        monkeypatch.setattr(ac, name, call)
    monkeypatch.setattr(ac, "_linear_block_fwd_call", lambda *a: call(a[12]))  # (its workspace)
    monkeypatch.setattr(ac, "_linear_block_bwd_call", lambda *a: call(a[11]))
    monkeypatch.setattr(ac, "_on_gpu", lambda *a: None)
    monkeypatch.setattr(ac, "_stream", lambda s=None: ctypes.c_void_p(0))
    monkeypatch.setattr(ac, "_WS", {})
    return got


@pytest.mark.parametrize("recipe", [ac.FP8Recipe(block=True), ac.FP8Recipe(dynamic=True)])
def test_a_captured_call_keeps_its_own(handed, monkeypatch, recipe):
    capturing = [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    x = torch.zeros(16, 48, dtype=B16, requires_grad=True)
    w = torch.zeros(32, 48, dtype=B16, requires_grad=True)
    for _ in range(2):
        with ac.fp8_autocast(recipe=recipe):
            y = ac.fp8_linear(x, w)
        y.backward(torch.zeros(16, 32, dtype=B16))
        assert not ac._WS, "kept beyond the capture"
    assert len(handed) == 4
    assert len({ws.data_ptr() for ws, _ in handed}) == 4
    if recipe.dynamic:
        assert not any(control.any() for _, control in handed), "control block not cleared"
    # an eager call on the same stream afterwards does not get a graph's memory
    capturing[0] = False
    with ac.fp8_autocast(recipe=recipe), torch.no_grad():
        ac.fp8_linear(x, w)
    assert handed[4][0].data_ptr() not in {ws.data_ptr() for ws, _ in handed[:4]}
    assert not handed[4][1].any()
