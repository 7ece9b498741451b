"""One tensor-parallel MLP block on the library's calls, trained with 8-bit
activations and served with 4-bit weights.

    y          = the norm before the block (left by the block before this one)
    u_k        = y W1_k                       column-parallel FC1, p shards
    h_k        = GeLU(u_k)
    b          = sum_k h_k W2_k               row-parallel FC2 and its AllReduce
    x_out, y'  = block_norm(x, b)             norm after, gate, residual, next norm

`MLPBlock.forward` keeps y and u_k in 8 bits, `backward` uses them; `QuantMLPBlock`
runs the same block for a few tokens with W1 and W2 in 4 bits.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

import torch

from . import tpfuse as tp


class MLPBlock:
    """bf16 weights: W1[k] [H, F] (column shards), W2[k] [F, H] (row shards);
    norm weights and gate as `tpfuse.block_norm` takes them (w_pre is the next
    block's norm)."""

    def __init__(self, W1: List[torch.Tensor], W2: List[torch.Tensor], w_pre: torch.Tensor, w_post: torch.Tensor,
                 gate: Optional[torch.Tensor] = None, alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
                 unit_offset: bool = False):
        self.W1, self.W2 = list(W1), list(W2)
        self.norm = dict(w_pre=w_pre, w_post=w_post, gate=gate, alpha=alpha, beta=beta, unit_offset=unit_offset)
        self.eps = eps

    def forward(self, x: torch.Tensor, y: torch.Tensor):
        """(x_out, y_next, kept): `kept` goes to `backward`."""
        _, y_codes, y_scales = tp.stash_pack([y], gelu=False)
        u = [tp.matmul_allreduce([y], [w]) for w in self.W1]
        h, u_codes, u_scales = tp.stash_pack(u, gelu=True)
        del u
        b = tp.matmul_allreduce(list(h), self.W2)
        x_out, y_next, stats = tp.block_norm(x, [b], eps=self.eps, want_stats=True, **self.norm)
        return x_out, y_next, (y_codes[0], y_scales[0], u_codes, u_scales, b, x_out, stats)

    def backward(self, dy_next: torch.Tensor, dx_out: Optional[torch.Tensor], kept):
        """Gradients by name: x, y (bf16), W1 and W2 (lists, fp32), w_pre, w_post, gate."""
        y_codes, y_scales, u_codes, u_scales, b, x_out, stats = kept
        dx, db, dw_pre, dw_post, dgate = tp.block_norm_backward(dy_next, dx_out, x_out, [b], stats, **self.norm)
        p = len(self.W1)
        dh = tp.rowpar_dx(db, self.W2)
        du, h = tp.stash_backward(u_codes, u_scales, dh)
        dW2 = tp.weight_grad(list(h), [db] * p)
        dW1 = tp.stash_weight_grad([y_codes] * p, [y_scales] * p, list(du))
        dy = tp.matmul_dx(list(du), self.W1)
        return {"x": dx, "y": dy, "W1": dW1, "W2": dW2, "w_pre": dw_pre, "w_post": dw_post, "gate": dgate}


def quantize(w: torch.Tensor, group: int = 128):
    """(codes, scales, zeros) of a weight [N, K] in the layout of
    `tpfuse.qweight_matmul`: 16 steps between each group's extremes (or zero)."""
    N, K = w.shape
    g = w.float().view(N, K // group, group)
    lo, hi = g.amin(2).clamp(max=0.0), g.amax(2).clamp(min=0.0)
    scales = ((hi - lo) / 15.0).clamp(min=2.0 ** -100).to(torch.bfloat16)
    s = scales.float()
    zeros = torch.round(-lo / s).clamp(0, 15)
    q = (torch.round(g / s[..., None]) + zeros[..., None]).clamp(0, 15).to(torch.uint8).view(N, K // 8, 2, 4)
    codes = (q[:, :, 0] | (q[:, :, 1] << 4)).reshape(N, K // 2)
    return codes.contiguous(), scales.contiguous(), zeros.to(torch.uint8).contiguous()


class QuantMLPBlock:
    """`MLPBlock` with 4-bit weights, for the few rows of a decode step."""

    def __init__(self, block: MLPBlock, group: int = 128):
        self.group, self.norm, self.eps = group, block.norm, block.eps
        self.W1 = [quantize(w.t(), group) for w in block.W1]                    # [F, H]
        self.W2 = list(zip(*(quantize(w.t(), group) for w in block.W2)))        # [H, F]: codes, scales, zeros

    def step(self, x: torch.Tensor, y: torch.Tensor, in_place: bool = True):
        """(x_out, y_next); the residual stream is updated in place by default."""
        h = [tp.qweight_matmul([y], [c], [s], [z], group=self.group, gelu=True) for c, s, z in self.W1]
        codes, scales, zeros = self.W2
        b = tp.qweight_matmul(h, codes, scales, zeros, group=self.group, out_dtype=torch.float32)
        x_out, y_next, _ = tp.block_norm(x, [b], eps=self.eps, x_out=x if in_place else None, **self.norm)
        return x_out, y_next


def example(tokens: int = 1024, H: int = 1024, F: int = 512, p: int = 4, steps: int = 3) -> Sequence[float]:
    """A few training steps on one batch, then a decode step; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, std=1.0):
        return torch.randn(shape, device="cuda", generator=g) * std

    block = MLPBlock([rand(H, F, std=H ** -0.5).bfloat16() for _ in range(p)],
                     [rand(F, H, std=F ** -0.5).bfloat16() for _ in range(p)],
                     torch.ones(H, device="cuda"), torch.ones(H, device="cuda"), torch.ones(H, device="cuda"))
    x, y, target = rand(tokens, H).bfloat16(), rand(tokens, H).bfloat16(), rand(tokens, H)
    losses = []
    for _ in range(steps):
        x_out, y_next, kept = block.forward(x, y)
        diff = y_next.float() - target
        losses.append(diff.square().mean())
        grads = block.backward((2.0 / tokens * diff).bfloat16(), None, kept)
        for name, params in (("W1", block.W1), ("W2", block.W2)):
            for w, dw in zip(params, grads[name]):
                w.copy_(w.float() - 0.05 * dw)
        for name in ("w_pre", "w_post", "gate"):
            block.norm[name] -= 0.05 * grads[name]
    QuantMLPBlock(block).step(x[:16].clone(), y[:16].contiguous())
    return [float(v) for v in losses]


if __name__ == "__main__":
    print("losses:", " ".join(f"{v:.4f}" for v in example()))
