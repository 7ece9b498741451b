"""One tensor-parallel MLP block of experts on the library's calls, with a shared
MLP beside them, its products in 8 bits.

    y          = the norm before the block (left by the block before this one)
    route      = the k experts of each token, from the logits y Wr
    u_k        = y W1_k[e]^T                  column-parallel FC1 of each token's experts, p shards
    h_k        = GeLU(u_k)
    b          = sum over a token's experts of weight * sum_k h_k W2_k[e]^T
    c          = the same of the shared MLP, V1 and V2, for every token
    x_out, y'  = block_norm(x, b + c)         norm after, gate, residual, next norm

`ExpertBlock.forward` keeps y, u_k and the experts' rows, `backward` uses them;
`step` runs the block for the few tokens of a decode step.

Precision: experts' and shared products have operands in 8 bits, and bf16 results
that the 8-bit matrix instructions sum (`tpfuse.fp8_matmul`); their weight gradients
are fp32.  The router's logits are fp32 sums of bf16 products; their gradient, fp32
as well, is rounded to bf16 (2^-9 of each value) before the products that give Wr's
and y's gradients, whose operands are bf16 as all the block's other gradients are.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

import torch

from . import tpfuse as tp

_F8 = torch.float8_e4m3fn


def quantize(w: torch.Tensor):
    """(codes, scales) of weights [..., N, K] as `tpfuse.fp8_matmul` and
    `tpfuse.expert_matmul` take them: e4m3, and for each 128 x 128 the exponent byte
    of the least power of two that keeps the block within e4m3's 448."""
    n, k = -w.shape[-2] % tp.SCALE_BLOCK, -w.shape[-1] % tp.SCALE_BLOCK
    blocks = torch.nn.functional.pad(w.detach().abs(), (0, k, 0, n)).unflatten(-1, (-1, tp.SCALE_BLOCK))
    top = blocks.unflatten(-3, (-1, tp.SCALE_BLOCK)).amax((-3, -1)).double()
    part, e = torch.frexp(top / 448.0)                     # part in [0.5, 1): 0.5 is a power of two itself
    e = torch.where(top > 0, e - (part == 0.5).int(), -117).clamp(-117, 127)
    each = e.repeat_interleave(tp.SCALE_BLOCK, -2).repeat_interleave(tp.SCALE_BLOCK, -1)
    codes = torch.ldexp(w.detach().float(), -each[..., :w.shape[-2], :w.shape[-1]]).to(_F8)
    return codes, (e + 127).to(torch.uint8)


def _turned(codes: torch.Tensor, scales: torch.Tensor):
    """The transposed weight: the blocks of 128 x 128 are its own."""
    return codes.view(torch.uint8).transpose(-1, -2).contiguous().view(_F8), scales.transpose(-1, -2).contiguous()


def _all(fn, ws):
    """Lists of codes and of scales over the shards."""
    return tuple(map(list, zip(*(fn(*w) if isinstance(w, tuple) else fn(w) for w in ws))))


class _MLP:
    """FC1, GeLU, FC2 in 8 bits: the experts' with a route, one for every token without."""

    def __init__(self, W1, W2):
        self.W1, self.W2 = list(W1), list(W2)
        self.requantize()

    def requantize(self):
        self.w1, self.w2 = _all(quantize, self.W1), _all(quantize, self.W2)
        self.w1t, self.w2t = _all(_turned, zip(*self.w1)), _all(_turned, zip(*self.w2))

    @staticmethod
    def product(x, xs, w, ws, route, **how):
        return tp.fp8_matmul(x, xs, w, ws, **how) if route is None else tp.expert_matmul(x, xs, w, ws, route, **how)

    @staticmethod
    def weight_grad(a, b, route):
        return tp.fp8_weight_grad(*a, *b) if route is None else tp.expert_weight_grad(*a, *b, route)

    def fc1(self, y, ys, route, **how):
        if route is not None:
            how["gather"] = True
        return [self.product([y], [ys], [w], [ws], route, **how) for w, ws in zip(*self.w1)]

    def fc2(self, h, route):
        codes, scales, _, _ = tp.fp8_pack(h)
        return self.product(codes, scales, *self.w2, route)

    def forward(self, y, ys, route):
        h, codes, scales = tp.stash_pack(self.fc1(y, ys, route), gelu=True)
        return self.fc2(list(h), route), (codes, scales)

    def backward(self, d, y, kept, route):
        """(gradient of the rows FC1 read, dW1, dW2) from d, the gradient of FC2's rows."""
        p = len(self.W1)
        dc, ds, dct, dst = tp.fp8_pack([d], columns=True, route=route)
        dh = [self.product(dc, ds, [w], [ws], route) for w, ws in zip(*self.w2t)]
        du, h = tp.stash_backward(*kept, dh)
        _, _, ht, hst = tp.fp8_pack(list(h), rows=False, columns=True, route=route)
        dW2 = self.weight_grad((list(dct) * p, list(dst) * p), (ht, hst), route)
        uc, us, uct, ust = tp.fp8_pack(list(du), columns=True, route=route)
        _, _, yt, yst = tp.fp8_pack([y], rows=False, columns=True, route=route, gather=route is not None)
        dW1 = self.weight_grad((uct, ust), (list(yt) * p, list(yst) * p), route)
        return self.product(uc, us, *self.w1t, route), dW1, dW2


class ExpertBlock:
    """bf16 weights: Wr [H, E]; W1[k] [E, F, H] (column shards) and W2[k] [E, H, F]
    (row shards) of the experts; V1[k] [Fs, H] and V2[k] [H, Fs] of the shared MLP,
    or none; norm weights and gate as `tpfuse.block_norm` takes them; score, bias,
    groups, renorm and scale as `tpfuse.expert_route` does.  `requantize` after a
    change of the weights."""

    def __init__(self, Wr: torch.Tensor, W1: List[torch.Tensor], W2: List[torch.Tensor], k: int, w_pre: torch.Tensor,
                 w_post: torch.Tensor, gate: Optional[torch.Tensor] = None, V1: Sequence[torch.Tensor] = (),
                 V2: Sequence[torch.Tensor] = (), alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
                 unit_offset: bool = False, score: str = "softmax", bias: Optional[torch.Tensor] = None,
                 groups: int = 1, top_groups: int = 1, renorm: bool = True, scale: float = 1.0):
        self.Wr, self.k, self.eps = Wr, k, eps
        self.experts, self.shared = _MLP(W1, W2), _MLP(V1, V2) if len(V1) else None
        self.norm = dict(w_pre=w_pre, w_post=w_post, gate=gate, alpha=alpha, beta=beta, unit_offset=unit_offset)
        self.weighing = dict(score=score, renorm=renorm, scale=scale)
        self.choosing = dict(bias=bias, groups=groups, top_groups=top_groups)

    def requantize(self):
        self.experts.requantize()
        if self.shared:
            self.shared.requantize()

    def route(self, y: torch.Tensor, mask: Optional[torch.Tensor] = None):
        """(logits [T, E] fp32, route); tokens whose `mask` is false go to no expert."""
        logits = tp.matmul_allreduce([y], [self.Wr], out_dtype=torch.float32)
        return logits, tp.expert_route(logits, self.k, mask=mask, **self.choosing, **self.weighing)

    def forward(self, x: torch.Tensor, y: torch.Tensor, mask: Optional[torch.Tensor] = None):
        """(x_out, y_next, kept): `kept` goes to `backward`."""
        logits, route = self.route(y, mask)
        (codes,), (scales,), _, _ = tp.fp8_pack([y])
        rows, u = self.experts.forward(codes, scales, route)
        b, v = [tp.expert_combine(rows, route)], None
        if self.shared:
            c, v = self.shared.forward(codes, scales, None)
            b.append(c)
        x_out, y_next, stats = tp.block_norm(x, b, eps=self.eps, want_stats=True, **self.norm)
        return x_out, y_next, (y, logits, route, rows, u, v, b, x_out, stats)

    def backward(self, dy_next: torch.Tensor, dx_out: Optional[torch.Tensor], kept):
        """Gradients by name: x, y (bf16), Wr (fp32), W1 and W2, V1 and V2 (lists, fp32), w_pre, w_post, gate."""
        y, logits, route, rows, u, v, b, x_out, stats = kept
        dx, db, dw_pre, dw_post, dgate = tp.block_norm_backward(dy_next, dx_out, x_out, b, stats, **self.norm)
        drows, dweights = tp.expert_combine_backward(db, rows, route)
        dlogits = tp.expert_route_backward(dweights, logits, route, **self.weighing).bfloat16()     # as the products take it
        dWr, = tp.weight_grad([y], [dlogits])
        dyr, dW1, dW2 = self.experts.backward(drows, y, u, route)
        dy = tp.expert_combine(dyr, route._replace(weights=torch.ones_like(route.weights)), out_dtype=torch.float32)
        dy += tp.matmul_dx([dlogits], [self.Wr], out_dtype=torch.float32)
        dV1, dV2 = [], []
        if self.shared:
            dys, dV1, dV2 = self.shared.backward(db, y, v, None)
            dy += dys
        return {"x": dx, "y": dy.bfloat16(), "Wr": dWr, "W1": dW1, "W2": dW2, "V1": dV1, "V2": dV2,
                "w_pre": dw_pre, "w_post": dw_post, "gate": dgate}

    def step(self, x: torch.Tensor, y: torch.Tensor, mask: Optional[torch.Tensor] = None, in_place: bool = True):
        """(x_out, y_next) of a few tokens; the residual stream is updated in place by default."""
        _, route = self.route(y, mask)
        (codes,), (scales,), _, _ = tp.fp8_pack([y])
        b = [tp.expert_combine(self.experts.fc2(self.experts.fc1(codes, scales, route, gelu=True), route), route)]
        if self.shared:
            b.append(self.shared.fc2(self.shared.fc1(codes, scales, None, gelu=True), None))
        x_out, y_next, _ = tp.block_norm(x, b, eps=self.eps, x_out=x if in_place else None, **self.norm)
        return x_out, y_next


def example(tokens: int = 1024, H: int = 1024, F: int = 512, E: int = 16, k: int = 4, p: int = 2,
            steps: int = 3) -> Sequence[float]:
    """A few training steps on one batch, then a decode step; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, std=1.0):
        return torch.randn(shape, device="cuda", generator=g) * std

    def shards(*shape, std):
        return [rand(*shape, std=std).bfloat16() for _ in range(p)]

    ones = [torch.ones(H, device="cuda") for _ in range(3)]
    block = ExpertBlock(rand(H, E, std=H ** -0.5).bfloat16(), shards(E, F, H, std=H ** -0.5),
                        shards(E, H, F, std=F ** -0.5), k, *ones, V1=shards(F, H, std=H ** -0.5),
                        V2=shards(H, F, std=F ** -0.5))
    x, y, target = rand(tokens, H).bfloat16(), rand(tokens, H).bfloat16(), rand(tokens, H)
    losses = []
    for _ in range(steps):
        x_out, y_next, kept = block.forward(x, y)
        diff = y_next.float() - target
        losses.append(diff.square().mean())
        grads = block.backward((2.0 / tokens * diff).bfloat16(), None, kept)
        for name, params in (("Wr", [block.Wr]), ("W1", block.experts.W1), ("W2", block.experts.W2),
                             ("V1", block.shared.W1), ("V2", block.shared.W2)):
            for w, dw in zip(params, [grads[name]] if name == "Wr" else grads[name]):
                w.copy_(w.float() - 0.05 * dw)
        for name in ("w_pre", "w_post", "gate"):
            block.norm[name] -= 0.05 * grads[name]
        block.requantize()
    block.step(x[:16].clone(), y[:16].contiguous())
    return [float(v) for v in losses]


if __name__ == "__main__":
    print("losses:", " ".join(f"{v:.4f}" for v in example()))
