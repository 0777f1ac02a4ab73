"""Activations of fp32 inputs against 64 bits, to the roundings of
their formulas in fp32.  Silu and gelu by tanh, with u = 2^-24, half a step:

    E = exp(-|w|)          2 u (exp to one step), what |w| itself is off times |w|
    r = 1 / (1 + E)        E's share is below half: 1 u, the sum 1 u, the division 1 u
    P, 1 - P               r, and E r: at most 2 + 1 + 1 + 1 = 5 u, so 5 u for either
    w                      v for silu, exact; for gelu by tanh c v (1 + 0.044715 v^2): two
                           constants, three products and an fma, 6 u
    P' = P (1 - P) w'      the two and a product; w' = c (1 + 0.134145 v^2): two constants,
                           three products and an fma
    a = v P, a' = P + v P' a product; an fma

P's relative change is (1 - P) times w's change, and 1 - P's is P times it.  Where
exp's result is below the normal numbers, it may be 0: 2^-126 off.

Gelu, P(-a) = exp(-a^2 / 2) t Q(t) / 2 with t = 1 / (1 + 0.2475 a): t is 4 u off (a
constant, an fma, the reciprocal to one step), or 3 near a = 0, where t Q(t) changes by 3.3
times as much and less further on: 10 u; Q's last additions and t Q 4 u, the
exponential, to one step, and its product 3 u, v P 1 u; and the exponent, v^2 / 2, is off by
its own product, log2 e and the product with it: 3 u of it."""

import math

import pytest
import torch

import expert_block_ref as ref
from expert_block_ref import U

pytestmark = pytest.mark.gpu
KINDS = {"silu": 0, "gelu_tanh": 2}


@pytest.fixture(scope="module")
def lib():
    import fp8_tensor_scaled_amd as f
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return f


def definition(v, kind):
    """a(v), a'(v) in 64 bits and how far fp32 steps may be from them."""
    v = v.double()
    if kind == KINDS["silu"]:
        w, slope_w, off_w, more = v, torch.ones_like(v), 0.0, 1
    else:
        c = math.sqrt(8 / math.pi)
        w, slope_w = c * (v + 0.044715 * v ** 3), c * (1 + 3 * 0.044715 * v * v)
        off_w, more = 6 * U * w.abs(), 7
    p, rest, tiny = torch.sigmoid(w), torch.sigmoid(-w), 2.0 ** -126
    off_p, off_rest = 5 * U + off_w * rest, 5 * U + off_w * p
    d = p * rest * slope_w
    off_d = (off_p + off_rest + more * U) * d + 2 * tiny * slope_w
    a, slope = v * p, p + v * d
    return (a, slope, (off_p + U) * a.abs() + tiny * v.abs(),
            off_p * p + tiny + v.abs() * off_d + U * slope.abs())


def values():
    """Dense where the functions bend, out to where exp ends, and random ones."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.cat([torch.linspace(-20, 20, 40000, device="cuda"),
                   torch.linspace(-110, 110, 8000, device="cuda"),
                   torch.randn(15999, generator=gen, device="cuda"),
                   torch.tensor([0.0], device="cuda")])
    return x.reshape(1, -1)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", list(KINDS))
def test_values(lib, kind, gated):
    x, k = values(), KINDS[kind]
    cols = x.shape[1]
    want, _, off, _ = definition(x, k)
    if gated:
        up = torch.randn(1, cols, device="cuda")
        x, off = torch.cat([x, up], 1), off * up.double().abs() + U * (want * up).abs()
        want = want * up.double()
    y = torch.empty(1, cols, device="cuda")
    lib.fp8_act_fwd(x, 1, cols, k, gated, y)
    ref.assert_within(y, want, off + ref.half_step(want, torch.float32), kind)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", list(KINDS))
def test_gradients(lib, kind, gated):
    """At every finite code with steps that spread them over the bend, and the
    far ones out to exp's end."""
    k = KINDS[kind]
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    codes = codes[torch.isfinite(codes.view(torch.float8_e4m3fn).float())]
    codes = torch.nn.functional.pad(codes, (0, 256 - codes.numel()))
    scales = torch.logspace(-3, -0.6, 400, device="cuda")
    rows = scales.numel()
    v = codes.view(torch.float8_e4m3fn).float()[None] * scales[:, None]
    value, slope, off_value, off_slope = definition(v, k)
    gen = torch.Generator(device="cuda").manual_seed(8)
    g = torch.randn(rows, 256, generator=gen, device="cuda")
    g64 = g.double()
    x8, steps = codes.repeat(rows, 1), scales[:, None].repeat(1, 2)
    want, off = g64 * slope, g64.abs() * off_slope + U * (g64 * slope).abs()
    if gated:  # (up: other codes, with the same steps)
        up8 = codes[torch.randperm(256, generator=gen, device="cuda")]
        up = (up8.view(torch.float8_e4m3fn).float()[None] * scales[:, None]).double()
        x8 = torch.stack([x8, up8.repeat(rows, 1)], 1).reshape(rows, 512)
        steps = torch.stack([steps, steps], 1).reshape(rows, 4)
        want = torch.cat([want * up, g64 * value], 1)
        off = torch.cat([off * up.abs() + U * (g64 * slope * up).abs(),
                         g64.abs() * off_value + U * (g64 * value).abs()], 1)
    dx = torch.empty(rows, 256 * (1 + gated), device="cuda")
    lib.fp8_act_bwd(g, rows, 256, k, gated, x8.contiguous(), steps.contiguous(), dx)
    ref.assert_within(dx, want, off + ref.half_step(want, torch.float32), kind)


def test_gelu_values(lib):
    x = values()
    y = torch.empty_like(x)
    lib.fp8_act_fwd(x, 1, x.shape[1], 1, False, y)
    v = x.double()
    want = 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    off = (18 + 1.5 * v * v) * U * want.abs() + 2.0 ** -126 * v.abs()
    ref.assert_within(y, want, off + ref.half_step(want, torch.float32), "gelu")
