"""Captured layer steps keep their scratch: a warm-up on the capture's stream
before, and eager calls of larger shapes there after, leave every replay right
and are not written to by one."""

import pytest
import torch

from fp8_tensor_scaled_amd.autocast import FP8Recipe, fp8_autocast, fp8_linear

pytestmark = pytest.mark.gpu


def step(x, w, g, recipe):
    with fp8_autocast(recipe=recipe):
        y = fp8_linear(x, w)
    return [y.detach(), *torch.autograd.grad(y, [x, w], g)]


def inputs(M, N, K):
    r = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    return r(M, K).requires_grad_(), r(N, K).requires_grad_(), r(M, N)


@pytest.mark.parametrize("warm", [True, False])
@pytest.mark.parametrize("recipe", [FP8Recipe(block=True), FP8Recipe(dynamic=True)],
                         ids=["block", "tensor"])
def test_replays_after_larger_eager_calls(recipe, warm):
    torch.manual_seed(3)
    small, large = inputs(64, 256, 384), inputs(512, 768, 640)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        if warm:
            step(*small, recipe)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = step(*small, recipe)
        first = step(*large, recipe)  # before any replay
        s.synchronize()
        # what was freed is used again; nothing may write to it
        junk = [torch.full((1 << 18,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(16)]
        for _ in range(4):
            with torch.no_grad():
                small[0].copy_(torch.randn(64, 384, device="cuda"))
            graph.replay()
            s.synchronize()
            for a, b in zip(captured, step(*small, recipe)):
                assert torch.equal(a, b)
            for a, b in zip(first, step(*large, recipe)):
                assert torch.equal(a, b)
        assert all(bool((j == 0x5A).all()) for j in junk)
    torch.cuda.current_stream().wait_stream(s)
