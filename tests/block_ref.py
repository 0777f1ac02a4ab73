"""Plain 64-bit implementations of the block-scaled operators, for their
tests: numpy only, written from the formulas, nothing shared with the
library."""

import numpy as np

import workloads as wl

BLOCK = 128
FMAX = (448.0, 57344.0)


def groups(n):
    return -(-n // BLOCK)


def round_fp8(v, fmt):
    """fp8 value nearest to v (64 bits), ties to even, saturating; NaN stays."""
    mant, emin = (3, -6) if fmt == 0 else (2, -14)
    v = np.asarray(v, np.float64)
    with np.errstate(invalid="ignore"):
        a = np.minimum(np.abs(v), FMAX[fmt])
        e = np.frexp(np.where(a > 0, a, 1.0))[1] - 1
        unit = np.ldexp(1.0, np.maximum(e, emin) - mant)
        return np.where(np.isnan(v), np.nan, np.copysign(np.round(a / unit) * unit, v))


def decode(c, fmt):
    """fp8 codes (uint8) -> their values in 64 bits."""
    c = np.asarray(c, np.uint8).astype(np.int64)
    s = np.where(c & 0x80, -1.0, 1.0)
    if fmt == 0:
        e, m, bias, mb = (c >> 3) & 15, c & 7, 7, 3
        special = (c & 0x7F) == 0x7F
        spec = np.full(c.shape, np.nan)
    else:
        e, m, bias, mb = (c >> 2) & 31, c & 3, 15, 2
        special = e == 31
        spec = np.where(m == 0, np.inf, np.nan)
    v = np.where(e == 0, np.ldexp(m.astype(float), 1 - bias - mb),
                 np.ldexp(1.0 + m / 2.0 ** mb, e - bias))
    return s * np.where(special, spec, v)


def grow(step, rows, cols, br, bc):
    """A step for each value of a rows x cols matrix from one for each block."""
    return np.asarray(step)[np.arange(rows)[:, None] // br, np.arange(cols)[None, :] // bc]


SHAPE = {"row": (1, BLOCK), "col": (BLOCK, 1), "tile": (BLOCK, BLOCK)}


def quantize(x, kind, fmt, margin=0):
    """(code values, steps) of float32 values x [rows][cols]: the formula's
    own fp32 steps, reciprocal and product, then an exact rounding."""
    br, bc = SHAPE[kind]
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    gr, gc = -(-rows // br), -(-cols // bc)
    pad = np.zeros((gr * br, gc * bc), np.float32)
    pad[:rows, :cols] = np.where(np.isnan(x), 0, np.abs(x))
    amax = pad.reshape(gr, br, gc, bc).max(axis=(1, 3))
    r = np.float32(1.0) / np.float32(FMAX[fmt])
    step = np.maximum(amax * r * np.float32(2.0 ** -margin), np.float32(1e-12)).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        inv = (np.float32(1.0) / step).astype(np.float32)
        scaled = (x * grow(inv, rows, cols, br, bc)).astype(np.float32)
    return round_fp8(scaled.astype(np.float64), fmt), step


def product(a, b, sa, sb, bias=None):
    """(value, bound) of sum_k a[i,k] b[k,j] with steps sa [m][kb] and
    sb [kb][n] per group of 128 k.  The bound is what the arithmetic may be
    off before the last rounding: the fp8 matrix instruction adds the products of
    8 neighbouring k after cutting each 13 bits below the largest one's
    leading bit (7 * 2^-13 of the largest), and every fp32 operation rounds
    (128 in a group, three for the scaling and the running sum)."""
    m, k = a.shape
    n = b.shape[1]
    kb = groups(k)
    value, bound, mag = np.zeros((m, n)), np.zeros((m, n)), np.zeros((m, n))
    for g in range(kb):
        s = np.abs(np.outer(sa[:, g].astype(float), sb[g].astype(float)))
        sg = np.outer(sa[:, g].astype(float), sb[g].astype(float))
        ka = slice(g * BLOCK, min(k, (g + 1) * BLOCK))
        value += a[:, ka] @ b[ka] * sg
        mag += np.abs(a[:, ka]) @ np.abs(b[ka]) * s
        for k8 in range(ka.start, ka.stop, 8):
            ks = slice(k8, min(k8 + 8, ka.stop))
            big = np.zeros((m, n))
            for kk in range(ks.start, ks.stop):
                big = np.maximum(big, np.abs(np.outer(a[:, kk], b[kk])))
            bound += 7 * 2.0 ** -13 * big * s
    bound += (BLOCK + 3 * kb + 3) * 2.0 ** -24 * mag
    if bias is not None:
        value = value + bias
        bound = bound + 2.0 ** -24 * np.abs(value)
    return value, bound


def bf16_tolerance(r):
    """Half a bf16 ulp is at most 2^-8 / 2 of the value, subnormal spacing aside; both
    sides of a rounding that the bound moves over make it a whole one."""
    return 2.0 ** -8 * np.abs(r) + 2.0 ** -133


def check_close(bits, value, bound, what):
    y = wl.bf16_bits_to_f32(bits).astype(np.float64).reshape(value.shape)
    err = np.abs(y - value)
    tol = bf16_tolerance(value) + bound
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, first at "
                           f"{np.argwhere(bad)[0]}: {y[bad][0]} for {value[bad][0]}, "
                           f"tolerance {tol[bad][0]}")


def route(logits, top_k, renorm):
    """(ids, weights): the largest logits of each row, ties to the lowest
    index, and their softmax weights."""
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    p = np.exp(logits - logits.max(1, keepdims=True))
    w = np.take_along_axis(p / p.sum(1, keepdims=True), ids, 1)
    return ids, w / w.sum(1, keepdims=True) if renorm else w


def moe(x, router, w13, w2, top_k, renorm):
    """(out, bound, ids, weights) in 64 bits; w13 [E][2H][D] and w2 [E][D][H]
    are dequantized values.  The bound follows fp32 sums (gamma_n of the sum
    of magnitudes), activations kept to 16 bits of precision, and 2^-20 for
    the exponentials and weights."""
    t, d = x.shape
    h = w13.shape[1] // 2
    ids, w = route(x @ router.T, top_k, renorm)
    out, bound = np.zeros((t, d)), np.zeros((t, d))
    gd, gh = (d + 8) * 2.0 ** -24, (h + 8) * 2.0 ** -24
    for i in range(t):
        for j, e in enumerate(ids[i]):
            a, mag = w13[e] @ x[i], np.abs(w13[e]) @ np.abs(x[i])
            g, u = a[:h], a[h:]
            silu = g / (1 + np.exp(-g))
            act = silu * u
            ea = (1.1 * np.abs(u) * mag[:h] + np.abs(silu) * mag[h:]) * gd
            ea = ea + (2.0 ** -16 + 2.0 ** -20) * np.abs(act)
            out[i] += w[i, j] * (w2[e] @ act)
            m2 = np.abs(w2[e])
            bound[i] += w[i, j] * (m2 @ ea + (gh + 2.0 ** -20) * (m2 @ np.abs(act)))
    return out, bound, ids, w
