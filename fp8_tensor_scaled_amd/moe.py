"""Mixture-of-experts module over ``fp8_quantize_block`` and ``fp8_moe``.

``FP8MoE`` keeps the experts' weights as fp8 codes with a step for each
128 x 128 tile, quantized once when it is made, and answers a few tokens at a
time (decoding): router, top-k, gated experts and their weighted sum are one
library call.  It has no gradient; experts are trained as dense layers
(``FP8Linear`` under ``FP8Recipe(block=True)``) and brought here for serving.
"""

from __future__ import annotations

import torch

from . import (E4M3, E5M2, _groups, _stream, _stream_lock, fp8_moe, fp8_moe_workspace,
               fp8_quantize_block)

__all__ = ["FP8MoE"]

_MAX_TOKENS = 1024  # of one library call

_WS: dict = {}  # (device index, stream) -> workspace, zero when new


def _workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    if torch.cuda.is_current_stream_capturing():
        # Cleared within the graph, whose memory it is: every replay finds it
        # as its first use needs it, and no eager call finds it uncleared.
        return torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    key = (dev.index, _stream().value)  # (its lock is held: see _stream_lock)
    ws = _WS.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _WS[key] = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    return ws


def _tile_codes(w: torch.Tensor, fmt: int) -> tuple:
    """bf16 [E][rows][cols] -> (codes, steps); tiles end with their expert."""
    experts, rows, cols = w.shape
    codes = torch.empty((experts, rows, cols), dtype=torch.uint8, device=w.device)
    steps = torch.empty((experts, _groups(rows), _groups(cols)), dtype=torch.float32,
                        device=w.device)
    for e in range(experts):
        fp8_quantize_block(w[e], rows, cols, fmt, out_tile=codes[e], scale_tile=steps[e])
    return codes, steps


class FP8MoE(torch.nn.Module):
    """router: bf16 [E][dim]; w13: bf16 [E][2 * hidden][dim], the gates' rows
    and then the up projections'; w2: bf16 [E][dim][hidden].  ``forward``
    takes bf16 [..., dim] and returns the same shape."""

    def __init__(self, router: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, top_k: int,
                 renormalize: bool = True, fmt: int = E4M3):
        super().__init__()
        for name, t, ndim in (("router", router, 2), ("w13", w13, 3), ("w2", w2, 3)):
            if t.dim() != ndim or t.dtype != torch.bfloat16 or not t.is_cuda:
                raise ValueError(f"FP8MoE: {name} must be a {ndim}-D bfloat16 tensor on the GPU")
        if fmt not in (E4M3, E5M2):
            raise ValueError(f"FP8MoE: bad format {fmt}")
        experts, dim = router.shape
        hidden = w2.shape[2]
        if (tuple(w13.shape) != (experts, 2 * hidden, dim)
                or tuple(w2.shape) != (experts, dim, hidden)):
            raise ValueError(f"FP8MoE: router {tuple(router.shape)}, w13 {tuple(w13.shape)} and "
                             f"w2 {tuple(w2.shape)} do not match")
        if not 1 <= top_k <= min(16, experts):
            raise ValueError(f"FP8MoE: top_k {top_k} outside [1, {min(16, experts)}]")
        if dim % 16 or hidden % 16:
            raise ValueError(f"FP8MoE: dim {dim} and hidden {hidden} must be multiples of 16")
        self.top_k, self.renormalize, self.fmt = int(top_k), bool(renormalize), fmt
        # (codes as uint8, which a module's .to(dtype) leaves alone; _apply keeps the rest)
        with torch.cuda.device(router.device):
            w13_codes, w13_steps = _tile_codes(w13.detach().contiguous(), fmt)
            w2_codes, w2_steps = _tile_codes(w2.detach().contiguous(), fmt)
        self.register_buffer("router", router.detach().clone().contiguous())
        self.register_buffer("w13", w13_codes)
        self.register_buffer("w13_steps", w13_steps)
        self.register_buffer("w2", w2_codes)
        self.register_buffer("w2_steps", w2_steps)

    def _apply(self, fn, recurse=True):
        """Moves follow the model; a conversion of its types (``.half()``,
        ``.to(torch.float32)``) leaves the router and the steps, whose types
        the library call asks for, as they were."""
        before = dict(self._buffers)
        super()._apply(fn, recurse)
        for name, old in before.items():
            new = self._buffers[name]
            if old is not None and new.dtype != old.dtype:
                self._buffers[name] = old.to(new.device)
        return self

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        experts, dim = self.router.shape
        if x.dtype != torch.bfloat16 or x.device != self.router.device or x.dim() < 1 \
                or x.shape[-1] != dim:
            raise ValueError(f"FP8MoE: input of shape {tuple(x.shape)}, {x.dtype} on {x.device}; "
                             f"expected bfloat16 [..., {dim}] on {self.router.device}")
        if torch.is_grad_enabled() and x.requires_grad:
            raise ValueError("FP8MoE: no gradient is defined; call it under torch.no_grad()")
        hidden = self.w2.shape[2]
        x2 = x.contiguous().reshape(-1, dim)
        if x2.data_ptr() % 16:  # a view that begins inside a buffer; the call wants whole 16 bytes
            x2 = x2.clone()
        out = torch.empty_like(x2)
        with torch.cuda.device(x.device):
            for at in range(0, x2.shape[0], _MAX_TOKENS):
                xs, ys = x2[at:at + _MAX_TOKENS], out[at:at + _MAX_TOKENS]
                n = xs.shape[0]
                need = fp8_moe_workspace(n, experts, self.top_k, dim, hidden)
                with _stream_lock(x.device, _stream()):
                    fp8_moe(xs, self.router, self.w13, self.w13_steps, self.w2, self.w2_steps, n,
                            experts, self.top_k, dim, hidden, self.fmt, self.renormalize,
                            _workspace(x.device, need), ys)
        return out.reshape(x.shape)
