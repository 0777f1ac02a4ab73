"""Autograd layer over the operators between an expert block's products, and
the block itself.

* ``fp8_layer_norm`` / ``FP8LayerNorm``: layer norm over the last dimension.
* ``fp8_activation``: silu or gelu, gated or not.  Inside an fp8_autocast region
  its input is kept for the backward as fp8 codes with a step for each 128
  values (in the region's forward format; the steps from the current amax
  whatever the recipe, without a margin), about half the memory of a 16-bit
  input; outside it is torch's own computation.
* ``fp8_sort_tokens``, ``fp8_dispatch``, ``fp8_combine``: tokens into their
  experts' order and back, weighted.
* ``FP8Experts``, ``FP8ExpertBlock``: gated experts for training, made of these
  and of ``FP8Linear`` layers, and the residual block around them; ``served()``
  gives the ``FP8MoE`` of the trained weights.

Every number is computed in libfp8lin (the entry points of __init__ that the
functions are named after); this module allocates outputs, reshapes, and keeps
what a backward needs.  Inputs are bf16, fp16 or fp32; each gradient has its
input's type.  Gradients are defined once: a second derivative raises.
"""

from __future__ import annotations

import contextlib
import math
from typing import NamedTuple

import torch

from . import (ACT_GELU, ACT_GELU_TANH, ACT_SILU, E4M3, _current_device, _groups, fp8_act_bwd,
               fp8_act_fwd, fp8_layer_norm_bwd, fp8_layer_norm_bwd_workspace, fp8_layer_norm_fwd,
               fp8_moe_combine, fp8_moe_combine_bwd, fp8_moe_dispatch, fp8_moe_sort,
               fp8_moe_sort_workspace)
from .autocast import FP8Linear, _once, current_config
from .moe import FP8MoE

__all__ = ["fp8_layer_norm", "FP8LayerNorm", "fp8_activation", "TokenOrder", "fp8_sort_tokens",
           "fp8_dispatch", "fp8_combine", "FP8Experts", "FP8ExpertBlock"]

_ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH}


def _on(t: torch.Tensor):
    """The tensor's device as the current one, whose stream the calls take."""
    if t.get_device() == _current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _gpu(who: str, **tensors) -> None:
    """All tensors on one GPU, of a type that the kernels take."""
    dev = next(iter(tensors.values())).device
    for name, t in tensors.items():
        if t is not None and (t.device.type != "cuda" or t.device != dev):
            raise ValueError(f"{who}: {name} is on {t.device}: all tensors must be on one GPU")


def _rows(t: torch.Tensor) -> tuple:
    """t [..., cols] as a matrix and its row stride, a copy only where the rows
    are not evenly spaced lines."""
    cols = t.shape[-1]
    m = t.reshape(math.prod(t.shape[:-1]), cols)
    if m.is_contiguous():
        return m, cols
    if m.stride(1) == 1 and m.stride(0) >= cols:
        return m, m.stride(0)
    return m.contiguous(), cols


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x2, ld = _rows(x)
        rows, cols = x2.shape
        y = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
        stats = torch.empty((2, rows), dtype=torch.float32, device=x.device)
        with _on(x):
            fp8_layer_norm_fwd(x2, rows, cols, weight, bias, eps, out=y, mean=stats[0],
                               rstd=stats[1], ldx=ld)
        ctx.save_for_backward(x2, weight, stats)
        ctx.conf = (ld, x.shape, None if bias is None else bias.dtype)
        return y.reshape(x.shape)

    @staticmethod
    @_once
    def backward(ctx, g):
        x2, weight, stats = ctx.saved_tensors
        ld, shape, bias_type = ctx.conf
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        rows, cols = x2.shape
        g2, ldg = _rows(g)
        dev = g.device
        dx = torch.empty((rows, cols), dtype=x2.dtype, device=dev) if need_x else None
        dw = torch.empty(cols, dtype=weight.dtype, device=dev) if need_w else None
        db = torch.empty(cols, dtype=bias_type, device=dev) if need_b else None
        ws = None
        if need_w or need_b:
            ws = torch.empty(fp8_layer_norm_bwd_workspace(rows, cols), dtype=torch.uint8,
                             device=dev)
        with _on(g):
            fp8_layer_norm_bwd(g2, x2, rows, cols, weight, stats[0], stats[1], dx, dw, db, ws,
                               ldg=ldg, ldx=ld)
        return None if dx is None else dx.reshape(shape), dw, db, None


def fp8_layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
                   bias: torch.Tensor | None = None, eps: float = 1e-5) -> torch.Tensor:
    """Layer norm of x [..., cols] over its last dimension.  weight, bias:
    [cols], of x's dtype or float32 (both the same)."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"fp8_layer_norm: input of shape {tuple(x.shape)}")
    for name, p in (("weight", weight), ("bias", bias)):
        if p is not None and (p.dim() != 1 or p.shape[0] != x.shape[-1]):
            raise ValueError(f"fp8_layer_norm: {name} of shape {tuple(p.shape)} for "
                             f"{x.shape[-1]} columns")
    _gpu("fp8_layer_norm", input=x, weight=weight, bias=bias)
    return _LayerNorm.apply(x, None if weight is None else weight.contiguous(),
                            None if bias is None else bias.contiguous(), float(eps))


class FP8LayerNorm(torch.nn.LayerNorm):
    """nn.LayerNorm over the last dimension through ``fp8_layer_norm``."""

    def __init__(self, normalized_shape, *args, **kw):
        super().__init__(normalized_shape, *args, **kw)
        if len(self.normalized_shape) != 1:
            raise ValueError("FP8LayerNorm: the norm is over the last dimension only (got "
                             f"{tuple(self.normalized_shape)})")

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.dim() < 1 or x.shape[-1] != self.normalized_shape[0]:
            raise ValueError(f"FP8LayerNorm: input of shape {tuple(x.shape)} for "
                             f"{self.normalized_shape[0]} columns")
        return fp8_layer_norm(x, self.weight, self.bias, self.eps)


class _Activation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, act, gated, fmt, grad_enabled):
        x2, ld = _rows(x)
        rows, halves = x2.shape[0], 2 if gated else 1
        cols = x2.shape[1] // halves
        y = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
        x8 = steps = None
        if grad_enabled and ctx.needs_input_grad[0]:
            x8 = torch.empty((rows, halves * cols), dtype=torch.uint8, device=x.device)
            steps = torch.empty((rows, halves * _groups(cols)), dtype=torch.float32,
                                device=x.device)
        with _on(x):
            fp8_act_fwd(x2, rows, cols, act, gated, y, x8=x8, steps=steps, fmt=fmt, ldx=ld)
        ctx.save_for_backward(x8, steps)
        ctx.conf = (cols, act, gated, fmt, x.shape)
        return y.reshape(*x.shape[:-1], cols)

    @staticmethod
    @_once
    def backward(ctx, g):
        x8, steps = ctx.saved_tensors
        cols, act, gated, fmt, shape = ctx.conf
        g2, ldg = _rows(g)
        dx = torch.empty(x8.shape, dtype=g.dtype, device=g.device)
        with _on(g):
            fp8_act_bwd(g2, g2.shape[0], cols, act, gated, x8, steps, dx, fmt=fmt, ldg=ldg)
        return dx.reshape(shape), None, None, None, None


def _torch_activation(x: torch.Tensor, kind: str) -> torch.Tensor:
    if kind == "silu":
        return torch.nn.functional.silu(x)
    return torch.nn.functional.gelu(x, approximate="tanh" if kind == "gelu_tanh" else "none")


def fp8_activation(x: torch.Tensor, kind: str = "silu", gated: bool = False) -> torch.Tensor:
    """``kind`` ("silu", "gelu", "gelu_tanh") of x [..., cols], or, gated, of
    the first half of x [..., 2 * cols] times the second.  Inside an
    fp8_autocast region the backward works from x in 8 bits (codes in the
    region's forward format); outside, this is torch's own computation."""
    if kind not in _ACTS:
        raise ValueError(f"fp8_activation: kind {kind!r}, expected one of {sorted(_ACTS)}")
    if x.dim() < 1 or (gated and x.shape[-1] % 2):
        raise ValueError(f"fp8_activation: input of shape {tuple(x.shape)}"
                         + (" cannot be halved" if gated else ""))
    cfg = current_config()
    if not cfg.enabled:
        if not gated:
            return _torch_activation(x, kind)
        gate, up = x.chunk(2, dim=-1)
        return _torch_activation(gate, kind) * up
    _gpu("fp8_activation", input=x)
    return _Activation.apply(x, _ACTS[kind], bool(gated), cfg.fp8_format.fwd(),
                             torch.is_grad_enabled())


class TokenOrder(NamedTuple):
    """The experts' order of a batch's (token, choice) pairs, fp8_moe_sort's:
    expert e has rows offsets[e] .. offsets[e + 1] - 1; slots [tokens][top_k] is
    each pair's row."""
    offsets: torch.Tensor
    slots: torch.Tensor
    experts: int


def fp8_sort_tokens(ids: torch.Tensor, experts: int) -> TokenOrder:
    """ids: [..., top_k] int32 or int64; an id outside [0, experts) is a pair of
    no expert."""
    if ids.dim() < 1 or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"fp8_sort_tokens: ids of shape {tuple(ids.shape)}, {ids.dtype}; "
                         "expected int32 or int64 [..., top_k]")
    _gpu("fp8_sort_tokens", ids=ids)
    top_k = ids.shape[-1]
    if ids.dtype == torch.int64:
        ids = ids.clamp(-1, experts).to(torch.int32)
    ids = ids.contiguous()
    tokens = math.prod(ids.shape[:-1])
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=ids.device)
    slots = torch.empty((tokens, top_k), dtype=torch.int32, device=ids.device)
    need = fp8_moe_sort_workspace(tokens, top_k, experts)
    ws = torch.empty(need, dtype=torch.uint8, device=ids.device) if need else None
    with _on(ids):
        fp8_moe_sort(ids, tokens, top_k, experts, offsets, slots, workspace=ws)
    return TokenOrder(offsets, slots, experts)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offsets, slots, experts):
        x2, ld = _rows(x)
        (tokens, dim), top_k = x2.shape, slots.shape[1]
        rows = torch.empty((tokens * top_k, dim), dtype=x.dtype, device=x.device)
        with _on(x):
            fp8_moe_dispatch(x2, tokens, top_k, dim, experts, offsets, slots, rows, ldx=ld)
        ctx.save_for_backward(offsets, slots)
        ctx.conf = (experts, x.shape)
        return rows

    @staticmethod
    @_once
    def backward(ctx, g):
        offsets, slots = ctx.saved_tensors
        experts, shape = ctx.conf
        tokens, top_k = slots.shape
        g = g.contiguous()
        dx = torch.empty((tokens, g.shape[1]), dtype=g.dtype, device=g.device)
        with _on(g):
            fp8_moe_combine(g, tokens, top_k, g.shape[1], experts, offsets, slots, None, dx)
        return dx.reshape(shape), None, None, None


def _check_order(who: str, order: TokenOrder, tokens: int) -> None:
    if order.slots.shape[0] != tokens:
        raise ValueError(f"{who}: {tokens} tokens, the order has {order.slots.shape[0]}")


def fp8_dispatch(x: torch.Tensor, order: TokenOrder) -> torch.Tensor:
    """x [..., dim] as rows [tokens * top_k][dim] in the experts' order; rows of
    no expert are zeros."""
    if x.dim() < 1:
        raise ValueError("fp8_dispatch: input of shape ()")
    _gpu("fp8_dispatch", input=x, slots=order.slots, offsets=order.offsets)
    _check_order("fp8_dispatch", order, math.prod(x.shape[:-1]))
    return _Dispatch.apply(x, order.offsets, order.slots, order.experts)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, offsets, slots, experts):
        (tokens, top_k), dim = slots.shape, rows.shape[1]
        out = torch.empty((tokens, dim), dtype=rows.dtype, device=rows.device)
        with _on(rows):
            fp8_moe_combine(rows, tokens, top_k, dim, experts, offsets, slots, weights, out)
        ctx.save_for_backward(rows if ctx.needs_input_grad[1] else None, weights, offsets, slots)
        ctx.experts = experts
        return out

    @staticmethod
    @_once
    def backward(ctx, g):
        rows, weights, offsets, slots = ctx.saved_tensors
        need_rows, need_weights = ctx.needs_input_grad[:2]
        tokens, top_k = slots.shape
        g2, ldg = _rows(g)
        dim = g2.shape[1]
        drows = dweights = None
        if need_rows:
            drows = torch.empty((tokens * top_k, dim), dtype=g.dtype, device=g.device)
        if need_weights:
            dweights = torch.empty((tokens, top_k), dtype=torch.float32, device=g.device)
        with _on(g):
            if weights is None:
                fp8_moe_dispatch(g2, tokens, top_k, dim, ctx.experts, offsets, slots, drows,
                                 ldx=ldg)
            else:
                fp8_moe_combine_bwd(g2, rows, tokens, top_k, dim, ctx.experts, offsets, slots,
                                    weights, drows, dweights, ldg=ldg)
        return drows, dweights, None, None, None


def fp8_combine(rows: torch.Tensor, order: TokenOrder,
                weights: torch.Tensor | None = None) -> torch.Tensor:
    """out [tokens][dim]: each token's rows, added up with fp32 weights
    [..., top_k] (or ones)."""
    if rows.dim() != 2 or rows.shape[0] != order.slots.numel():
        raise ValueError(f"fp8_combine: rows of shape {tuple(rows.shape)} for "
                         f"{order.slots.numel()} pairs")
    if weights is not None:
        if weights.dtype != torch.float32 or weights.numel() != order.slots.numel() \
                or weights.shape[-1:] != order.slots.shape[1:]:
            raise ValueError(f"fp8_combine: weights of shape {tuple(weights.shape)}, "
                             f"{weights.dtype}; expected float32 [..., {order.slots.shape[1]}] "
                             f"for {order.slots.shape[0]} tokens")
        weights = weights.reshape(order.slots.shape).contiguous()
    _gpu("fp8_combine", rows=rows, weights=weights, slots=order.slots, offsets=order.offsets)
    return _Combine.apply(rows.contiguous(), weights, order.offsets, order.slots, order.experts)


class FP8Experts(torch.nn.Module):
    """Gated experts as they are trained: a router, then for each token its
    top_k experts, weighted by the softmax of their logits (over the chosen
    ones with ``renormalize``, over all without).  Each expert is two
    ``FP8Linear`` layers around a gated silu, and takes its tokens as one run of
    rows; one without tokens takes no part in the batch, and its weights get no
    gradient (None, not zeros).  ``forward`` takes bf16 [..., dim]; it waits for the
    tokens' counts (they are sizes of what follows), so it cannot be captured into a
    graph."""

    def __init__(self, dim: int, hidden: int, experts: int, top_k: int, renormalize: bool = True,
                 device=None, dtype=torch.bfloat16):
        super().__init__()
        if not 1 <= top_k <= min(16, experts) or experts > 512:
            raise ValueError(f"FP8Experts: top_k {top_k} of {experts} experts; expected 1 .. "
                             f"{min(16, experts)} of at most 512")
        kw = dict(device=device, dtype=dtype)
        self.top_k, self.renormalize = int(top_k), bool(renormalize)
        self.router = torch.nn.Parameter(torch.randn(experts, dim, **kw) * dim ** -0.5)
        self.up = torch.nn.ModuleList(FP8Linear(dim, 2 * hidden, bias=False, **kw)
                                      for _ in range(experts))
        self.down = torch.nn.ModuleList(FP8Linear(hidden, dim, bias=False, **kw)
                                        for _ in range(experts))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        experts = len(self.up)
        if x.is_cuda and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("FP8Experts: the tokens' counts are read on the host, so a call "
                               "cannot be captured into a graph")
        logits = x.float() @ self.router.float().t()
        if self.renormalize:
            top, ids = logits.topk(self.top_k, dim=-1)
            weights = top.softmax(-1)
        else:
            weights, ids = logits.softmax(-1).topk(self.top_k, dim=-1)
        order = fp8_sort_tokens(ids, experts)
        rows = fp8_dispatch(x, order)
        at = order.offsets.tolist() + [rows.shape[0]]
        parts = list(rows.split([b - a for a, b in zip(at, at[1:])]))
        for e in range(experts):
            if parts[e].shape[0]:
                hidden = fp8_activation(self.up[e](parts[e]), "silu", gated=True)
                parts[e] = self.down[e](hidden)
        return fp8_combine(torch.cat(parts), order, weights).reshape(x.shape)

    def served(self, fmt: int = E4M3) -> FP8MoE:
        """The same experts with their weights as tile-scaled codes, for a few
        tokens at a time."""
        return FP8MoE(self.router, torch.stack([m.weight for m in self.up]),
                      torch.stack([m.weight for m in self.down]), self.top_k, self.renormalize,
                      fmt)


class FP8ExpertBlock(torch.nn.Module):
    """x + experts(norm(x))."""

    def __init__(self, dim: int, hidden: int, experts: int, top_k: int, renormalize: bool = True,
                 eps: float = 1e-5, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.norm = FP8LayerNorm(dim, eps=eps, device=device, dtype=dtype)
        self.experts = FP8Experts(dim, hidden, experts, top_k, renormalize, device, dtype)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return x + self.experts(self.norm(x))
