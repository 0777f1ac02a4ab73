"""Operands, outputs and weights whose offsets pass 31 and 32 bits, checked on
rows and columns at their ends."""

import numpy as np
import pytest
import torch

from tests import block_ref as href
from tests import block_ref_gpu as ref

pytestmark = pytest.mark.gpu
E4M3 = 0


@pytest.fixture(scope="module")
def f():
    import fp8_tensor_scaled_amd as f
    return f


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def ends(n, seed, count=40):
    rng = np.random.default_rng(seed)
    i = np.concatenate([[0, 1, n - 2, n - 1], n - 1 - rng.integers(0, min(n, 300), count // 2),
                        rng.integers(0, n, count // 2)])
    return torch.from_numpy(np.unique(i)).cuda()


def codes(rows, cols, seed):
    """Random codes without NaN, made in place (no wider copy)."""
    c = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    c.random_(0, 0x7F, generator=ref.generator(seed))
    c[:, ::3] |= 0x80
    return c


@pytest.mark.parametrize("layout,m,n,k", [
    ("nt", 131100, 48, 16400),    # A past 2^31 bytes
    ("nn", 40, 140000, 16400),    # B past 2^31 bytes, columns contiguous
    ("tn", 16400, 64, 262200),    # A past 2^32 bytes, rows along k
    ("nt", 66000, 66064, 144),    # an output past 2^32 elements, tiled
])
def test_products(f, layout, m, n, k):
    ta, tb, G = int(layout[0] == "t"), int(layout[1] == "t"), ref.groups
    a = codes(*((k, m) if ta else (m, k)), 1)
    b = codes(*((n, k) if tb else (k, n)), 2)
    tile_b = layout != "tn"
    sa = ref.steps(*((G(k), m) if ta else (m, G(k))), seed=3)
    lines = G(n) if tile_b else n
    sb = ref.steps(*((lines, G(k)) if tb else (G(k), lines)), seed=4)
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    f.fp8_mm_block(a, b, E4M3, E4M3, ta, tb, m, n, k, m if ta else k, k if tb else n, sa,
                   f.GROUP_LINE, sb, f.GROUP_TILE if tile_b else f.GROUP_LINE, None, out)
    i, j = ends(m, 5), ends(n, 6)
    av = ref.decode(a[:, i].t().contiguous() if ta else a[i], E4M3)
    bv = ref.decode(b[j].t().contiguous() if tb else b[:, j].contiguous(), E4M3)
    jg = j // 128 if tile_b else j
    ref.check_close(out[i][:, j], *ref.product(av, bv, sa[:, i].t() if ta else sa[i],
                                               sb[jg].t() if tb else sb[:, jg]), layout)


@pytest.mark.parametrize("kinds", [("row", "col"), ("tile",)])
def test_quantize(f, kinds):
    rows, cols = 66003, 65536 + 200  # 4.3e9 elements
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=ref.generator(1))
    G = ref.groups
    shape = {"row": (rows, G(cols)), "col": (G(rows), cols), "tile": (G(rows), G(cols))}
    got = {k: (torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
               torch.empty(*shape[k], device="cuda")) for k in kinds}
    f.fp8_quantize_block(x, rows, cols, E4M3, **{"out_" + k: v[0] for k, v in got.items()},
                         **{"scale_" + k: v[1] for k, v in got.items()})
    r0, c0 = G(rows) * 128 - 256, G(cols) * 128 - 256  # the last tiles, and some in the middle
    for r, c in ((0, 0), (r0, c0), (r0, 0), (0, c0), (32768, 65536 - 128)):
        part = x[r:r + 256, c:c + 256].float().cpu().numpy()
        h, w = part.shape
        for kind, (q, s) in got.items():
            want, steps = href.quantize(part, kind, E4M3)
            br, bc = href.SHAPE[kind]
            sub = s[r // br:r // br + steps.shape[0], c // bc:c // bc + steps.shape[1]]
            np.testing.assert_array_equal(sub.cpu().numpy(), steps)
            np.testing.assert_array_equal(href.decode(q[r:r + h, c:c + w].cpu().numpy(), E4M3),
                                          want)


@pytest.mark.parametrize("t", [1, 3])
def test_experts(f, t):
    """Weights past 2^32 bytes: the last experts are the chosen ones."""
    e, k, d, h = 64, 3, 4096, 8208
    w13 = codes(e * 2 * h, d, 1).view(e, 2 * h, d)
    w2 = codes(e * d, h, 2).view(e, d, h)
    G = ref.groups
    s13 = ref.steps(e, G(2 * h), G(d), seed=3) * 1e-3
    s2 = ref.steps(e, G(d), G(h), seed=4) * 1e-3
    x = torch.randn(t, d, device="cuda", generator=ref.generator(5)).bfloat16()
    router = torch.zeros(e, d, device="cuda").bfloat16()
    for i, expert in enumerate((63, 61, 0)):  # their logits are the largest for every token
        router[expert] = (x.float().mean(0).sign() * (3 - i) * 0.02).bfloat16()
    out = torch.empty(t, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(t, k, dtype=torch.int32, device="cuda")
    ws = torch.zeros(f.fp8_moe_workspace(t, e, k, d, h), dtype=torch.uint8, device="cuda")
    f.fp8_moe(x, router, w13, s13, w2, s2, t, e, k, d, h, E4M3, True, ws, out, ids=ids)
    host = lambda v: v.float().cpu().numpy().astype(np.float64)  # noqa: E731
    assert set(ids.flatten().tolist()) == {63, 61, 0}
    used = [0, 61, 63]
    w13v = np.stack([host(ref.decode(w13[i], E4M3)) * href.grow(host(s13[i]), 2 * h, d, 128, 128)
                     for i in used])
    w2v = np.stack([host(ref.decode(w2[i], E4M3)) * href.grow(host(s2[i]), d, h, 128, 128)
                    for i in used])
    # the other experts' logits are 0: softmax over all, renormalized over the chosen
    want, bound, wids, _ = href.moe(host(x), host(router[used]), w13v, w2v, k, True)
    assert np.array_equal(np.array(used)[wids], ids.cpu().numpy())
    got = out.view(torch.int16).cpu().numpy().view(np.uint16)
    href.check_close(got, want, bound, f"{t} tokens")
