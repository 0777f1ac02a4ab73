"""The block-scaled product and expert layer in 64 bits with elementary torch
operations on the GPU: block_ref.py's formulas and bounds for outputs too many
for the host."""

import numpy as np
import torch

BLOCK = 128
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
FMAX = (448.0, 57344.0)


def groups(n):
    return -(-n // BLOCK)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(rows, cols, fmt, seed):
    """fp8 codes (uint8) [rows][cols]: a bell that reaches the largest value."""
    v = torch.randn(rows, cols, device="cuda", generator=generator(seed)) * (FMAX[fmt] / 4)
    return v.clamp_(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)


def steps(*shape, seed):
    return torch.exp(torch.randn(*shape, device="cuda", generator=generator(seed))) * 0.01


def decode(c, fmt):
    return c.view(F8[fmt]).float()


def product(a, b, sa, sb, bias=None):
    """(value, bound) of sum_k a[i,k] b[k,j] with steps sa [m][kb] and sb
    [kb][n]: what block_ref.product gives, in its terms."""
    m, k = a.shape
    n = b.shape[1]
    kb = groups(k)
    value, bound, mag = (torch.zeros(m, n, device=a.device, dtype=torch.float64)
                         for _ in range(3))
    for g in range(kb):
        s = torch.outer(sa[:, g].double(), sb[g].double())
        ag = a[:, g * BLOCK:(g + 1) * BLOCK].double().contiguous()
        bg = b[g * BLOCK:(g + 1) * BLOCK].double().contiguous()
        value += torch.mm(ag, bg) * s
        mag += torch.mm(ag.abs(), bg.abs()) * s.abs()
        cut = torch.zeros(m, n, device=a.device, dtype=torch.float64)
        af, bf = ag.abs().float(), bg.abs().float()  # (products of two codes are exact)
        for k8 in range(0, ag.shape[1], 8):
            big = torch.zeros(m, n, device=a.device)
            for kk in range(k8, min(k8 + 8, ag.shape[1])):
                big = torch.maximum(big, af[:, kk, None] * bf[None, kk])
            cut += big
        bound += 7 * 2.0 ** -13 * cut * s.abs()
    bound += (BLOCK + 3 * kb + 3) * 2.0 ** -24 * mag
    if bias is not None:
        value = value + bias.double()
        bound = bound + 2.0 ** -24 * value.abs()
    return value, bound


def check_close(got, value, bound, what):
    """Every output of bf16 `got` within the bound and the rounding to bf16."""
    err = (got.double().reshape(value.shape) - value).abs()
    tol = 2.0 ** -8 * value.abs() + 2.0 ** -133 + bound
    bad = ~(err <= tol)
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {at}: "
                             f"{got.reshape(value.shape)[at].item()} for {value[at].item()}, "
                             f"tolerance {tol[at].item()}")


class Operands:
    """A product's operands as stored for a layout, and as matrices."""

    def __init__(self, layout, m, n, k, fa, fb, tile_a, tile_b, bias, seed):
        self.ta, self.tb = int(layout[0] == "t"), int(layout[1] == "t")
        ta, tb, G = self.ta, self.tb, groups
        self.a = codes(*((k, m) if ta else (m, k)), fa, seed)
        self.b = codes(*((n, k) if tb else (k, n)), fb, seed + 1)
        lm, ln = (G(m) if tile_a else m), (G(n) if tile_b else n)
        self.sa = steps(*((G(k), lm) if ta else (lm, G(k))), seed=seed + 2)
        self.sb = steps(*((ln, G(k)) if tb else (G(k), ln)), seed=seed + 3)
        self.bias = (torch.randn(n, device="cuda", generator=generator(seed + 4)) * 5).bfloat16() \
            if bias else None
        self.args = (fa, fb, ta, tb, m, n, k, m if ta else k, k if tb else n)
        self.groups = (int(tile_a), int(tile_b))
        self.shape = (m, n, k)

    def matrices(self):
        m, n, k = self.shape
        fa, fb = self.args[:2]
        a, b = decode(self.a, fa), decode(self.b, fb)
        sa = self.sa.t() if self.ta else self.sa
        sb = self.sb.t() if self.tb else self.sb
        if self.groups[0]:
            sa = sa.repeat_interleave(BLOCK, 0)[:m]
        if self.groups[1]:
            sb = sb.repeat_interleave(BLOCK, 1)[:, :n]
        return a.t() if self.ta else a, b.t() if self.tb else b, sa, sb

    def check(self, outs, what):
        """Each of the outputs against the definition."""
        value, bound = product(*self.matrices(), self.bias)
        for out in outs:
            check_close(out, value, bound, what)

    def run(self, f, workspace=None, pad=64):
        """The library's output; what lies behind it stays as it was."""
        m, n, _ = self.shape
        out = torch.full((m * n + pad,), 0x7A11, dtype=torch.int16, device="cuda")
        f.fp8_mm_block(self.a, self.b, *self.args, self.sa, self.groups[0], self.sb,
                       self.groups[1], self.bias, out, workspace=workspace)
        assert bool((out[m * n:] == 0x7A11).all()), "output overrun"
        return out[:m * n].view(torch.bfloat16).reshape(m, n)


def bits_equal(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def to_host(t):
    return t.detach().cpu().numpy().astype(np.float64)
