"""Two threads on the default stream, which shares one workspace per kind of
call: each gets the bits of the same calls made by one thread."""

import threading

import pytest
import torch

from fp8_tensor_scaled_amd.autocast import FP8Recipe, fp8_autocast, fp8_linear
from fp8_tensor_scaled_amd.moe import FP8MoE

pytestmark = pytest.mark.gpu
REPEATS = 40


def normal(*shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std).bfloat16()


def experts(e, d, h, k, tokens, seed):
    m = FP8MoE(normal(e, d, seed=seed, std=d ** -0.5),
               normal(e, 2 * h, d, seed=seed + 1, std=d ** -0.5),
               normal(e, d, h, seed=seed + 2, std=h ** -0.5), k)
    x = normal(tokens, d, seed=seed + 3)

    def call():
        with torch.no_grad():
            return [m(x)]
    return call


def layer(M, N, K, recipe, seed):
    x = normal(M, K, seed=seed).requires_grad_()
    w = normal(N, K, seed=seed + 1, std=0.02).requires_grad_()
    g = normal(M, N, seed=seed + 2)

    def call():
        with fp8_autocast(recipe=recipe):
            y = fp8_linear(x, w)
        return [y.detach(), *torch.autograd.grad(y, [x, w], g)]
    return call


def check(*calls):
    want = [c() for c in calls]
    torch.cuda.synchronize()
    start, results, errors = threading.Barrier(len(calls)), [[] for _ in calls], []

    def run(i):
        try:
            start.wait()
            for _ in range(REPEATS):
                results[i].append(calls[i]())
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i, w in enumerate(want):
        assert len(results[i]) == REPEATS
        for got in results[i]:
            assert all(torch.equal(a, b) for a, b in zip(got, w)), i


def test_experts_of_two_shapes():
    check(experts(16, 256, 128, 4, 13, 1), experts(6, 144, 80, 2, 40, 9))


def test_block_layers_of_two_shapes():
    r = FP8Recipe(block=True)
    check(layer(256, 384, 256, r, 1), layer(64, 1024, 512, r, 9))


@pytest.mark.parametrize("recipe", [FP8Recipe(dynamic=True), FP8Recipe()],
                         ids=["dynamic", "delayed"])
def test_block_layer_beside_a_tensor_scaled_one(recipe):
    check(layer(256, 384, 256, FP8Recipe(block=True), 1), layer(64, 1024, 512, recipe, 9))
