"""The expert module and the example that trains and serves experts."""

import os
import runpy

import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def module():
    from fp8_tensor_scaled_amd.moe import FP8MoE
    return FP8MoE


def weights(e, d, h, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return ((r(e, d) * d ** -0.5).bfloat16(), (r(e, 2 * h, d) * d ** -0.5).bfloat16(),
            (r(e, d, h) * h ** -0.5).bfloat16())


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def values(w, fmt):
    out = []
    for e in range(w.shape[0]):
        q, s = ref.quantize(host(w[e]), "tile", fmt)
        out.append(q * ref.grow(s, *w.shape[1:], 128, 128))
    return np.stack(out)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("shape", [(1,), (3, 5), (0,), (40,)])
def test_against_the_definition(module, shape, fmt):
    e, k, d, h = 6, 2, 144, 80
    router, w13, w2 = weights(e, d, h, 3)
    m = module(router, w13, w2, k, fmt=fmt)
    x = torch.randn(*shape, d, device="cuda").bfloat16()
    y = m(x)
    assert y.shape == x.shape and y.dtype == torch.bfloat16
    if x.numel() == 0:
        return
    out, bound, _, _ = ref.moe(host(x).reshape(-1, d), host(router), values(w13, fmt),
                               values(w2, fmt), k, True)
    bits = y.reshape(-1, d).view(torch.int16).cpu().numpy().view(np.uint16)
    ref.check_close(bits, out, bound, f"{shape} {fmt}")


def test_more_tokens_than_a_call_takes(module):
    """Rows of a long input have the bits of a call on their own part."""
    m = module(*weights(4, 64, 32, 5), 2)
    x = torch.randn(2100, 64, device="cuda").bfloat16()
    y = m(x)
    for at in (0, 1024, 2048):
        assert torch.equal(y[at:at + 1024], m(x[at:at + 1024]))


def test_strided_input_state_and_streams(module):
    m = module(*weights(4, 64, 32, 7), 3, renormalize=False)
    wide = torch.randn(9, 96, device="cuda").bfloat16()
    x = wide[:, 16:80]
    y = m(x)
    assert torch.equal(y, m(x.contiguous()))
    other = module(*weights(4, 64, 32, 8), 3, renormalize=False)
    other.load_state_dict(m.state_dict())
    assert torch.equal(y, other(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        z = m(x)
    s.synchronize()
    assert torch.equal(y, z)


def test_captured_first(module):
    """The first call of a shape may be a captured one; replays and eager
    calls between them have the same bits."""
    m = module(*weights(8, 128, 256, 9), 4)
    x = torch.randn(11, 128, device="cuda").bfloat16()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y = m(x)
    for _ in range(4):
        x.copy_(torch.randn(11, 128, device="cuda"))
        want = m(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_refusals(module):
    router, w13, w2 = weights(4, 64, 32, 11)
    for args, kw, needle in (((router.float(), w13, w2, 2), {}, "router"),
                             ((router, w13[0], w2, 2), {}, "w13"),
                             ((router, w13, w2.cpu(), 2), {}, "w2"),
                             ((router, w13[:, :32], w2, 2), {}, "do not match"),
                             ((router, w13, w2[:3], 2), {}, "do not match"),
                             ((router, w13, w2, 0), {}, "top_k"),
                             ((router, w13, w2, 5), {}, "top_k"),
                             ((router, w13, w2, 2), dict(fmt=2), "format"),
                             ((router[:, :60], w13[..., :60], w2[:, :60], 2), {}, "multiples")):
        with pytest.raises(ValueError, match=needle):
            module(*args, **kw)
    m = module(router, w13, w2, 2)
    good = torch.randn(3, 64, device="cuda").bfloat16()
    for x in (good.float(), good.cpu(), good[:, :32]):
        with pytest.raises(ValueError, match="expected bfloat16"):
            m(x)
    with pytest.raises(ValueError, match="no gradient"):
        m(good.requires_grad_())


def test_example():
    """Training lowers the loss; serving differs from the trained form by the
    rounding of two activations to E4M3 (each at most 2^-4 of a value, so at
    most 2^-4 of a gate, an up and a hidden value's size in the mean: below
    three times that of the norm)."""
    main = runpy.run_path(os.path.join(ROOT, "examples", "train_and_serve_experts.py"))["main"]
    r = main(steps=30, tokens=256, dim=128, hidden=160, experts=4, top_k=2, outputs=300)
    assert r["last"] < 0.9 * r["first"]
    for n in (1, 13, 64):
        assert r[n] < 3 * 2.0 ** -4
