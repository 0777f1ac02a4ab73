"""Workspaces that the autograd layers and the expert module keep per stream
(no GPU): threads share a stream (the default one is every thread's current
stream), and a library call is several launches that hand data on through the
workspace.  So no other thread may enqueue a call on it between the time a call
takes its workspace and the time all its launches are enqueued."""

import ctypes
import threading
import time

import pytest
import torch

from fp8_tensor_scaled_amd import autocast as ac
from fp8_tensor_scaled_amd import moe

B16 = torch.bfloat16


class Calls:
    """Stands for library calls: each takes a while, as a call whose launches
    the interpreter lock does not cover, and notes calls that overlap it."""

    def __init__(self, monkeypatch):
        self.inside, self.overlaps, self.made = 0, 0, 0
        for m in (ac, moe):
            monkeypatch.setattr(m, "_stream", lambda s=None: ctypes.c_void_p(0))
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        monkeypatch.setattr(ac, "_WS", {})
        monkeypatch.setattr(moe, "_WS", {})

    def __call__(self, *args, **kw):
        self.inside += 1
        self.made += 1
        self.overlaps += self.inside > 1
        time.sleep(0.01)
        self.inside -= 1

    def from_threads(self, *work):
        errors = []

        def run(w):
            try:
                for _ in range(4):
                    w()
            except BaseException as e:  # noqa: BLE001
                errors.append(e)

        threads = [threading.Thread(target=run, args=(w,)) for w in work]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not errors, errors
        assert self.made and not self.overlaps, f"{self.overlaps} of {self.made} calls overlapped"


@pytest.fixture
def calls(monkeypatch):
    return Calls(monkeypatch)


def layer(recipe, m, n, k, backward):
    def work():
        x = torch.zeros(m, k, dtype=B16, requires_grad=backward)
        w = torch.zeros(n, k, dtype=B16, requires_grad=backward)
        with ac.fp8_autocast(recipe=recipe):
            y = ac.fp8_linear(x, w)
        if backward:
            y.backward(torch.zeros(m, n, dtype=B16))
    return work


def test_block_layer(calls, monkeypatch):
    monkeypatch.setattr(ac, "_on_gpu", lambda *a: None)
    for name in ("_linear_block_fwd_call", "_linear_block_bwd_call"):
        monkeypatch.setattr(ac, name, calls)
    recipe = ac.FP8Recipe(block=True)
    calls.from_threads(layer(recipe, 16, 32, 48, True), layer(recipe, 160, 320, 480, True))


def test_tensor_scaled_layer(calls, monkeypatch):
    for name in ("_linear_fwd_call", "_linear_bwd_call"):
        monkeypatch.setattr(ac, name, calls)
    recipe = ac.FP8Recipe(dynamic=True)
    calls.from_threads(layer(recipe, 16, 32, 48, True), layer(recipe, 160, 320, 480, True))


def test_expert_module(calls, monkeypatch):
    monkeypatch.setattr(moe, "fp8_moe", calls)
    monkeypatch.setattr(torch.cuda, "device", lambda d: torch.no_grad())

    def module(experts, dim, hidden):
        m = moe.FP8MoE.__new__(moe.FP8MoE)
        torch.nn.Module.__init__(m)
        m.top_k, m.renormalize, m.fmt = 2, True, 0
        m.register_buffer("router", torch.zeros(experts, dim, dtype=B16))
        m.register_buffer("w13", torch.zeros(experts, 2 * hidden, dim, dtype=torch.uint8))
        m.register_buffer("w2", torch.zeros(experts, dim, hidden, dtype=torch.uint8))
        m.w13_steps = m.w2_steps = None
        return lambda: m(torch.zeros(3, dim, dtype=B16))

    calls.from_threads(module(4, 64, 32), module(8, 256, 128))
