"""Trains gated experts with block-scaled fp8 layers, then serves them.

Training: each expert is two ``FP8Linear`` layers under
``FP8Recipe(block=True)`` (E4M3 forward, E5M2 gradients, a step per 128
values), fitted to a random teacher.  Serving: an output head's weight is
quantized once by ``fp8_quantize_block``; a token goes through ``FP8MoE`` (the
trained experts as tile-scaled codes), and its result through
``fp8_quantize_block`` and ``fp8_mm_block`` to the head's outputs.

    python examples/train_and_serve_experts.py
"""

from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fp8_tensor_scaled_amd as fp8  # noqa: E402
from fp8_tensor_scaled_amd.autocast import (FP8Format, FP8Linear, FP8Recipe,  # noqa: E402
                                            fp8_autocast)
from fp8_tensor_scaled_amd.moe import FP8MoE  # noqa: E402


class Experts(torch.nn.Module):
    """The layer as it is trained: tokens gathered expert by expert."""

    def __init__(self, dim: int, hidden: int, experts: int, top_k: int):
        super().__init__()
        kw = dict(bias=False, device="cuda", dtype=torch.bfloat16)
        self.top_k = top_k
        self.router = torch.nn.Parameter(
            torch.randn(experts, dim, device="cuda", dtype=torch.bfloat16) * dim ** -0.5)
        self.up = torch.nn.ModuleList(FP8Linear(dim, 2 * hidden, **kw) for _ in range(experts))
        self.down = torch.nn.ModuleList(FP8Linear(hidden, dim, **kw) for _ in range(experts))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        logits = x.float() @ self.router.float().t()
        top, ids = logits.topk(self.top_k, dim=-1)
        weights = top.softmax(-1)  # over the chosen ones
        out = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        for e in range(len(self.up)):
            token, rank = (ids == e).nonzero(as_tuple=True)
            if token.numel() == 0:
                continue
            gate, up = self.up[e](x[token]).chunk(2, dim=-1)
            h = torch.nn.functional.silu(gate) * up
            y = self.down[e](h).float() * weights[token, rank, None]
            out = out.index_add(0, token, y)
        return out

    def served(self) -> FP8MoE:
        return FP8MoE(self.router, torch.stack([m.weight for m in self.up]),
                      torch.stack([m.weight for m in self.down]), self.top_k)


class Head:
    """y = x W^T on codes: x quantized by rows, W by tiles, once."""

    def __init__(self, weight: torch.Tensor):
        self.n, self.k = weight.shape
        tiles = [(s + 127) // 128 for s in weight.shape]
        self.codes = torch.empty(weight.shape, dtype=torch.uint8, device="cuda")
        self.steps = torch.empty(tiles, device="cuda")
        fp8.fp8_quantize_block(weight, self.n, self.k, fp8.E4M3, out_tile=self.codes,
                               scale_tile=self.steps)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        m = x.shape[0]
        x8 = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
        sx = torch.empty(m, (self.k + 127) // 128, device="cuda")
        y = torch.empty(m, self.n, dtype=torch.bfloat16, device="cuda")
        fp8.fp8_quantize_block(x, m, self.k, fp8.E4M3, out_row=x8, scale_row=sx)
        fp8.fp8_mm_block(x8, self.codes, fp8.E4M3, fp8.E4M3, 0, 1, m, self.n, self.k, self.k,
                         self.k, sx, fp8.GROUP_LINE, self.steps, fp8.GROUP_TILE, None, y)
        return y


def main(steps: int = 60, tokens: int = 512, dim: int = 256, hidden: int = 384,
         experts: int = 8, top_k: int = 2, outputs: int = 1000, seed: int = 0) -> dict:
    torch.manual_seed(seed)
    model = Experts(dim, hidden, experts, top_k)
    teacher = torch.randn(dim, dim, device="cuda") * dim ** -0.5
    optimizer = torch.optim.Adam(model.parameters(), lr=5e-3)
    recipe = FP8Recipe(block=True)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, dim, device="cuda", dtype=torch.bfloat16)
        with fp8_autocast(recipe=recipe, fp8_format=FP8Format.HYBRID):
            loss = (model(x) - x.float() @ teacher).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
        if step % 20 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {loss.item():.4f}", flush=True)

    serve = model.served()
    head = Head(torch.randn(outputs, dim, device="cuda", dtype=torch.bfloat16) * dim ** -0.5)
    result = dict(first=losses[0].item(), last=losses[-1].item())
    with torch.no_grad():
        for n in (1, 13, 64):
            x = torch.randn(n, dim, device="cuda", dtype=torch.bfloat16)
            with fp8_autocast(recipe=recipe, fp8_format=FP8Format.HYBRID):
                trained = model(x)
            y = serve(x)
            diff = ((y.float() - trained).norm() / trained.norm()).item()
            logits = head(y)
            result[n] = diff
            print(f"{n:3d} tokens: served against trained {diff:.4f} of the norm, "
                  f"first choice of token 0: {int(logits[0].argmax())}", flush=True)
    return result


if __name__ == "__main__":
    main()
