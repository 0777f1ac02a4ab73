"""The block-scaled fp8 operators as cases to be timed and compared.

Three operators and the training step made of them:

  quantize  fp8 codes with one step for each group of 128 values: along a row
            (1 x 128, activations), along a column (128 x 1, what a weight
            gradient contracts over) or for a 128 x 128 tile (weights)
  product   the matrix product of such operands, in the forward's (NT), the
            input gradient's (NN) and the weight gradient's (TN) layouts
  step      a linear layer's forward and backward with both
  moe       a whole mixture-of-experts layer for a few tokens: router, top-k,
            gated experts with tile-scaled weights, weighted sum

`run` computes them in elementary torch operations in 32 bits, or, with
`own`, by the package's entry points.
"""

import math

import torch

own = False

E4M3, E5M2 = 0, 1
FMAX = (448.0, 57344.0)
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 128
STEP_MIN = 1e-12


def listed():
    return [
        # the activations of 16 decoded tokens before a projection: latency
        dict(name="quantize_decode", op="quantize", rows=16, cols=2048, pad=0, kind="row",
             fmt=E4M3, dtype="bf16"),
        # fp16 activations of a training step, no size a multiple of 128, a
        # slice of a wider tensor: both groupings from one read
        dict(name="quantize_rowcol_ragged", op="quantize", rows=4111, cols=1000, pad=24,
             kind="rowcol", fmt=E4M3, dtype="f16"),
        # a large weight (the benchmark's 8192 x 8192): bandwidth
        dict(name="quantize_tile_8192", op="quantize", rows=8192, cols=8192, pad=0, kind="tile",
             fmt=E4M3, dtype="bf16"),
        # the benchmark's short product, 64 rows against an 8192 x 2048 weight
        dict(name="product_decode", op="product", layout="nt", m=64, n=8192, k=2048, fa=E4M3,
             fb=E4M3, tile_b=True, bias=False),
        # the benchmark's square product with a bias: matrix-core rate
        dict(name="product_4096", op="product", layout="nt", m=4096, n=4096, k=4096, fa=E4M3,
             fb=E4M3, tile_b=True, bias=True),
        # an input gradient where no side is a multiple of 16: rows start anywhere
        dict(name="product_dx_ragged", op="product", layout="nn", m=1000, n=1111, k=2047, fa=E5M2,
             fb=E4M3, tile_b=True, bias=False),
        # the weight gradient of the training configuration: steps along both
        # operands' columns
        dict(name="product_dw", op="product", layout="tn", m=4096, n=1024, k=2048, fa=E5M2,
             fb=E4M3, tile_b=False, bias=False),
        # the small linear layer: launches and host work count
        dict(name="step_256", op="step", m=256, n=256, k=256, fmt="e4m3", bias=True),
        # the training configuration's layer, E4M3 forward and E5M2 gradients
        dict(name="step_train", op="step", m=2048, n=4096, k=1024, fmt="hybrid", bias=True),
        # one decoded token, 8 of 64 experts
        dict(name="moe_1", op="moe", tokens=1, experts=64, top_k=8, dim=2048, hidden=1024,
             renorm=True, fmt=E4M3),
        # an odd batch, 2 of 32 experts, sides that are no multiple of 128
        dict(name="moe_13", op="moe", tokens=13, experts=32, top_k=2, dim=1040, hidden=688,
             renorm=False, fmt=E4M3),
        # 64 tokens that reach every expert: all weights are read
        dict(name="moe_64", op="moe", tokens=64, experts=64, top_k=8, dim=2048, hidden=1024,
             renorm=True, fmt=E4M3),
    ]


def _log(rng, lo, hi, mult=1):
    """A size spread over the logarithm of its range, a multiple of `mult`."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return _whole(max(lo, min(hi, v)), mult)


def _whole(v, mult):
    """v down to a multiple of `mult`; whole thousands (of 1024) only as powers of two."""
    v = max(mult, v // mult * mult)
    return v - mult if v % 1024 == 0 and v & (v - 1) else v


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "step", "moe", "moe"])
    if op == "quantize":
        rows, cols = _log(rng, 1, 8192), _log(rng, 16, 4096)
        if rng.random() < 0.5:
            cols = _whole(cols, 8)
        return dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 3, 24]),
                    kind=rng.choice(["row", "col", "rowcol", "tile"]),
                    fmt=rng.choice([E4M3, E5M2]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "product":
        m = _log(rng, 1, 4096)
        n, k = _log(rng, 128, 4096), _log(rng, 128, 4096)
        if rng.random() < 0.7:  # rows that a user lays out in whole 16 bytes
            n, k = _whole(n, 16), _whole(k, 16)
            m = _whole(m, 16) if m > 64 else m
        layout = rng.choice(["nt", "nt", "nn", "tn"])
        fa, fb = rng.choice([(E4M3, E4M3), (E5M2, E4M3), (E5M2, E5M2)])
        return dict(op=op, layout=layout, m=m, n=n, k=k, fa=fa, fb=fb,
                    tile_b=layout != "tn" and rng.random() < 0.8, bias=rng.random() < 0.5)
    if op == "step":
        return dict(op=op, m=_log(rng, 16, 2048, 16), n=_log(rng, 128, 2048, 16),
                    k=_log(rng, 128, 2048, 16), fmt=rng.choice(["e4m3", "hybrid"]),
                    bias=rng.random() < 0.5)
    experts = rng.choice([8, 16, 24, 32, 48, 64])
    dim, hidden = _log(rng, 256, 2048, 16), _log(rng, 128, 1024, 16)
    return dict(op=op, tokens=_log(rng, 1, 64), experts=experts,
                top_k=rng.choice([1, 2, 4, 6, 8]), dim=dim, hidden=hidden,
                renorm=rng.random() < 0.5, fmt=rng.choice([E4M3, E4M3, E5M2]))


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _codes(shape, fmt, gen):
    """fp8 codes as a block quantize leaves them: a bell whose ends reach the
    format's largest value."""
    v = torch.randn(shape, generator=gen, device="cuda") * (FMAX[fmt] / 4)
    return v.clamp_(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])


def _steps(shape, fmt, std, gen):
    """Steps of blocks whose values have about this deviation, each block's its own."""
    v = torch.randn(shape, generator=gen, device="cuda")
    return (std * 4 / FMAX[fmt]) * torch.exp(0.5 * v)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1009 + 17)
    c = case

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    if c["op"] == "quantize":
        rows, cols = c["rows"], c["cols"]
        # a few channels of activations are much larger than the others
        wide = torch.exp(torch.randn(1, cols + c["pad"], generator=gen, device="cuda"))
        x = (torch.randn(rows, cols + c["pad"], generator=gen, device="cuda") * wide)
        x = x.to(DTYPE[c["dtype"]])[:, :cols]
        f8 = F8[c["fmt"]]
        s = dict(case=c, x=x)
        if "row" in c["kind"]:
            s["row"] = torch.empty(rows, cols, dtype=f8, device="cuda")
            s["row_step"] = torch.empty(rows, _blocks(cols), device="cuda")
        if "col" in c["kind"]:
            s["col"] = torch.empty(rows, cols, dtype=f8, device="cuda")
            s["col_step"] = torch.empty(_blocks(rows), cols, device="cuda")
        if c["kind"] == "tile":
            s["tile"] = torch.empty(rows, cols, dtype=f8, device="cuda")
            s["tile_step"] = torch.empty(_blocks(rows), _blocks(cols), device="cuda")
        return s
    if c["op"] == "product":
        m, n, k, kb = c["m"], c["n"], c["k"], _blocks(c["k"])
        ta, tb = c["layout"][0] == "t", c["layout"][1] == "t"
        s = dict(case=c, a=_codes((k, m) if ta else (m, k), c["fa"], gen),
                 b=_codes((n, k) if tb else (k, n), c["fb"], gen))
        s["sa"] = _steps((kb, m) if ta else (m, kb), c["fa"], 1.0, gen)
        if c["tile_b"]:
            s["sb"] = _steps((_blocks(n), kb) if tb else (kb, _blocks(n)), c["fb"], 0.02, gen)
        else:
            s["sb"] = _steps((n, kb) if tb else (kb, n), c["fb"], 0.02, gen)
        s["bias"] = normal(n, std=0.1) if c["bias"] else None
        s["out"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        if own:
            import fp8_tensor_scaled_amd as f
            need = f.fp8_mm_block_workspace(m, n, k)
            s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
        return s
    if c["op"] == "step":
        m, n, k = c["m"], c["n"], c["k"]
        wide = torch.exp(0.5 * torch.randn(1, k, generator=gen, device="cuda"))
        x = (torch.randn(m, k, generator=gen, device="cuda") * wide).to(torch.bfloat16)
        return dict(case=c, x=x.requires_grad_(True),
                    w=normal(n, k, std=0.02).requires_grad_(True),
                    bias=normal(n, std=0.1).requires_grad_(True) if c["bias"] else None,
                    g=normal(m, n, std=1e-3))
    t, e, d, h = c["tokens"], c["experts"], c["dim"], c["hidden"]
    s = dict(case=c, x=normal(t, d), router=normal(e, d, std=1.5 / math.sqrt(d)))
    s["w13"] = _codes((e, 2 * h, d), c["fmt"], gen)
    s["s13"] = _steps((e, _blocks(2 * h), _blocks(d)), c["fmt"], 1 / math.sqrt(d), gen)
    s["w2"] = _codes((e, d, h), c["fmt"], gen)
    s["s2"] = _steps((e, _blocks(d), _blocks(h)), c["fmt"], 1 / math.sqrt(h), gen)
    s["out"] = torch.empty(t, d, dtype=torch.bfloat16, device="cuda")
    s["ids"] = torch.empty(t, c["top_k"], dtype=torch.int32, device="cuda")
    s["weights"] = torch.empty(t, c["top_k"], device="cuda")
    if own:
        import fp8_tensor_scaled_amd as f
        need = f.fp8_moe_workspace(t, e, c["top_k"], d, h)
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _run_own(s):
    import fp8_tensor_scaled_amd as f
    c = s["case"]
    if c["op"] == "quantize":
        f.fp8_quantize_block(s["x"], c["rows"], c["cols"], c["fmt"], out_row=s.get("row"),
                             scale_row=s.get("row_step"), out_col=s.get("col"),
                             scale_col=s.get("col_step"), out_tile=s.get("tile"),
                             scale_tile=s.get("tile_step"), ldx=c["cols"] + c["pad"])
        return {k: v for k, v in s.items() if k not in ("case", "x")}
    if c["op"] == "product":
        ta, tb = int(c["layout"][0] == "t"), int(c["layout"][1] == "t")
        m, n, k = c["m"], c["n"], c["k"]
        f.fp8_mm_block(s["a"], s["b"], c["fa"], c["fb"], ta, tb, m, n, k, m if ta else k,
                       k if tb else n, s["sa"], f.GROUP_LINE, s["sb"],
                       f.GROUP_TILE if c["tile_b"] else f.GROUP_LINE, s["bias"], s["out"],
                       workspace=s["ws"])
        return s["out"]
    if c["op"] == "step":
        from fp8_tensor_scaled_amd.autocast import FP8Recipe, fp8_autocast, fp8_linear
        with fp8_autocast(recipe=FP8Recipe(block=True), fp8_format=c["fmt"]):
            y = fp8_linear(s["x"], s["w"], s["bias"])
        ins = [s["x"], s["w"]] + ([s["bias"]] if c["bias"] else [])
        return [y.detach()] + list(torch.autograd.grad(y, ins, s["g"]))
    f.fp8_moe(s["x"], s["router"], s["w13"], s["s13"], s["w2"], s["s2"], c["tokens"],
              c["experts"], c["top_k"], c["dim"], c["hidden"], c["fmt"], c["renorm"], s["ws"],
              s["out"], ids=s["ids"], weights=s["weights"])
    return dict(out=s["out"], ids=s["ids"], weights=s["weights"])


def _pad_to(v, rows, cols):
    return torch.nn.functional.pad(v, (0, cols - v.shape[1], 0, rows - v.shape[0]))


def _quantize(x, kind, fmt):
    """Codes (fp8) and steps of x by groups of 128: step = max(amax / FMAX,
    1e-12), code = the fp8 value nearest to x * (1 / step), ties to even."""
    rows, cols = x.shape
    br, bc = {"row": (1, BLOCK), "col": (BLOCK, 1), "tile": (BLOCK, BLOCK)}[kind]
    gr, gc = (rows + br - 1) // br, (cols + bc - 1) // bc
    v = _pad_to(x.float(), gr * br, gc * bc).reshape(gr, br, gc, bc)
    step = torch.clamp_min(v.abs().amax(dim=(1, 3)) / FMAX[fmt], STEP_MIN)
    q = v * (1.0 / step)[:, None, :, None]
    q = q.clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).reshape(gr * br, gc * bc)
    return q[:rows, :cols].contiguous(), step


def _values(q, step, br, bc):
    """What codes with a step for each br x bc block stand for, in 32 bits."""
    s = step.repeat_interleave(br, -2) if br > 1 else step
    s = s.repeat_interleave(bc, -1) if bc > 1 else s
    return q.float() * s[..., :q.shape[-2], :q.shape[-1]]


def _route(logits, top_k, renorm):
    """The top_k experts of each token (ties to the lowest index) and their
    softmax weights."""
    order = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :top_k]
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    w = torch.gather(p / p.sum(1, keepdim=True), 1, order)
    return order, w / w.sum(1, keepdim=True) if renorm else w


def _moe_plain(s):
    c = s["case"]
    t, e, h = c["tokens"], c["experts"], c["hidden"]
    x = s["x"].float()
    ids, weights = _route(x @ s["router"].float().t(), c["top_k"], c["renorm"])
    if t * c["top_k"] <= e:  # the chosen experts' weights for each token
        at = ids.reshape(-1)
        w13 = _values(s["w13"][at], s["s13"][at], BLOCK, BLOCK)
        a = torch.bmm(w13, x.repeat_interleave(c["top_k"], 0)[:, :, None])[:, :, 0]
        a = torch.nn.functional.silu(a[:, :h]) * a[:, h:]
        w2 = _values(s["w2"][at], s["s2"][at], BLOCK, BLOCK)
        y = torch.bmm(w2, a[:, :, None])[:, :, 0].reshape(t, c["top_k"], -1)
        y = (y * weights[:, :, None]).sum(1)
    else:  # every expert for every token, weighted by zero where it was not chosen
        w13 = _values(s["w13"], s["s13"], BLOCK, BLOCK)
        a = torch.matmul(x[None], w13.transpose(1, 2))
        a = torch.nn.functional.silu(a[:, :, :h]) * a[:, :, h:]
        w2 = _values(s["w2"], s["s2"], BLOCK, BLOCK)
        dense = torch.zeros(t, e, device=x.device).scatter_(1, ids, weights)
        y = (torch.matmul(a, w2.transpose(1, 2)) * dense.t()[:, :, None]).sum(0)
    return dict(out=y.to(torch.bfloat16), ids=ids.to(torch.int32), weights=weights)


def _step_values(s, quantize, values, formats):
    """Output and gradients of the layer from quantized operands: x and w for
    y; g (along n) and w for dx; g and x (along the tokens) for dw."""
    ff, fb = formats
    c, x, w, g = s["case"], s["x"].detach(), s["w"].detach(), s["g"]
    wq = values(*quantize(w, "tile", ff), BLOCK, BLOCK)
    y = values(*quantize(x, "row", ff), 1, BLOCK) @ wq.t()
    dx = values(*quantize(g, "row", fb), 1, BLOCK) @ wq
    dw = values(*quantize(g, "col", fb), BLOCK, 1).t() @ values(*quantize(x, "col", ff), BLOCK, 1)
    return c, y, dx, dw


def _formats(name):
    return (E4M3, E5M2) if name == "hybrid" else (E4M3, E4M3)


def run(state):
    if own:
        return _run_own(state)
    s, c = state, state["case"]
    if c["op"] == "quantize":
        r = {}
        if "row" in c["kind"]:
            r["row"], r["row_step"] = _quantize(s["x"], "row", c["fmt"])
        if "col" in c["kind"]:
            r["col"], r["col_step"] = _quantize(s["x"], "col", c["fmt"])
        if c["kind"] == "tile":
            r["tile"], r["tile_step"] = _quantize(s["x"], "tile", c["fmt"])
        return r
    if c["op"] == "product":
        ta, tb = c["layout"][0] == "t", c["layout"][1] == "t"
        a = _values(s["a"], s["sa"], BLOCK if ta else 1, 1 if ta else BLOCK)
        if c["tile_b"]:
            b = _values(s["b"], s["sb"], BLOCK, BLOCK)
        else:
            b = _values(s["b"], s["sb"], 1 if tb else BLOCK, BLOCK if tb else 1)
        y = (a.t() if ta else a) @ (b.t() if tb else b)
        return (y if s["bias"] is None else y + s["bias"].float()).to(torch.bfloat16)
    if c["op"] == "step":
        c, y, dx, dw = _step_values(s, _quantize, _values, _formats(c["fmt"]))
        y = y + s["bias"].detach().float() if c["bias"] else y
        out = [y, dx, dw] + ([s["g"].float().sum(0)] if c["bias"] else [])
        return [v.to(torch.bfloat16) for v in out]
    return _moe_plain(s)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        rb, cb = _blocks(c["rows"]), _blocks(c["cols"])
        steps = {"row": c["rows"] * cb, "col": rb * c["cols"], "tile": rb * cb,
                 "rowcol": c["rows"] * cb + rb * c["cols"]}[c["kind"]]
        codes = 2 if c["kind"] == "rowcol" else 1
        return dict(bytes=n * (SIZE[c["dtype"]] + codes) + 4 * steps, flops=2 * n * codes)
    if c["op"] == "product":
        m, n, k, kb = c["m"], c["n"], c["k"], _blocks(c["k"])
        steps = m * kb + (_blocks(n) if c["tile_b"] else n) * kb
        return dict(bytes=m * k + n * k + 4 * steps + 2 * m * n + (2 * n if c["bias"] else 0),
                    flops=2 * m * n * k)
    if c["op"] == "step":
        m, n, k = c["m"], c["n"], c["k"]
        # x, w, g and the bias once; y, dx, dw and the bias' gradient once
        return dict(bytes=2 * (2 * m * k + 2 * n * k + 2 * m * n + (2 * n if c["bias"] else 0)),
                    flops=6 * m * n * k)
    t, e, k, d, h = c["tokens"], c["experts"], c["top_k"], c["dim"], c["hidden"]
    reached = e * (1.0 - (1.0 - k / e) ** t)  # experts that some token chose, on average
    per_expert = 3 * d * h + 4 * (_blocks(2 * h) * _blocks(d) + _blocks(d) * _blocks(h))
    return dict(bytes=int(reached * per_expert) + 2 * e * d + 4 * t * d + 8 * t * k,
                flops=2 * t * k * 3 * d * h + 2 * t * e * d)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _round_fp8(v, fmt):
    """The fp8 value nearest to v (ties to even), in 64 bits: multiples of
    2^(e - mantissa bits) in the binade [2^e, 2^(e+1)), down to the subnormal spacing."""
    bits, lowest = (3, -6) if fmt == E4M3 else (2, -14)
    e = torch.frexp(v)[1].to(torch.float64) - 1.0
    unit = torch.exp2(torch.clamp_min(e, float(lowest)) - bits)
    return (torch.round(v / unit) * unit).clamp(-FMAX[fmt], FMAX[fmt])


def _grow(step, rows, cols, br, bc):
    """A step for each value of a rows x cols matrix from one for each block."""
    i = torch.arange(rows, device=step.device) // br
    j = torch.arange(cols, device=step.device) // bc
    return step[..., i[:, None], j[None, :]]


def _quantize64(x, kind, fmt):
    br, bc = {"row": (1, BLOCK), "col": (BLOCK, 1), "tile": (BLOCK, BLOCK)}[kind]
    x = x.double()
    rows, cols = x.shape
    v = x.abs()
    if bc > 1:
        v = torch.stack([p.amax(1) for p in v.split(bc, 1)], 1)
    if br > 1:
        v = torch.stack([p.amax(0) for p in v.split(br, 0)], 0)
    step = torch.clamp_min(v / FMAX[fmt], STEP_MIN)
    return _round_fp8(x / _grow(step, rows, cols, br, bc), fmt), step


def _values64(q, step, br, bc):
    return q.double() * _grow(step.double(), q.shape[-2], q.shape[-1], br, bc)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "quantize":
        r = {}
        for kind in ("row", "col", "tile"):
            if kind in c["kind"]:
                r[kind], r[kind + "_step"] = _quantize64(s["x"], kind, c["fmt"])
        return r
    if c["op"] == "product":
        ta, tb = c["layout"][0] == "t", c["layout"][1] == "t"
        a = _values64(s["a"], s["sa"], BLOCK if ta else 1, 1 if ta else BLOCK)
        wide = BLOCK if c["tile_b"] else 1
        b = _values64(s["b"], s["sb"], wide if tb else BLOCK, BLOCK if tb else wide)
        y = torch.matmul(a.t() if ta else a, b.t() if tb else b)
        return y if s["bias"] is None else y + s["bias"].double()
    if c["op"] == "step":
        _, y, dx, dw = _step_values(s, _quantize64, _values64, _formats(c["fmt"]))
        if not c["bias"]:
            return [y, dx, dw]
        return [y + s["bias"].detach().double(), dx, dw, s["g"].double().sum(0)]
    h = c["hidden"]
    x = s["x"].double()
    logits = torch.matmul(x, s["router"].double().t())
    p = torch.softmax(logits, 1)
    weights, ids = [], []
    for t in range(c["tokens"]):
        row = sorted(range(c["experts"]), key=lambda e, r=logits[t].tolist(): (-r[e], e))
        ids.append(row[:c["top_k"]])
        weights.append(p[t, ids[-1]])
    weights = torch.stack(weights)
    if c["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(c["experts"]):
        hit = [(t, row.index(e)) for t, row in enumerate(ids) if e in row]
        if not hit:
            continue
        ts, js = [t for t, _ in hit], [j for _, j in hit]
        a = torch.matmul(x[ts], _values64(s["w13"][e], s["s13"][e], BLOCK, BLOCK).t())
        a = a[:, :h] / (1 + torch.exp(-a[:, :h])) * a[:, h:]
        o = torch.matmul(a, _values64(s["w2"][e], s["s2"][e], BLOCK, BLOCK).t())
        y[ts] += o * weights[ts, js][:, None]
    return dict(out=y, ids=torch.tensor(ids, dtype=torch.int32), weights=weights)
