"""The MLP block's operators in float64 on the CPU, written from their
definitions, with the sizes of the terms that each result is summed from
(the rounding errors of fp32 sums are proportional to those)."""
import math

import torch

D = torch.float64
STEP = 2.0 ** -24            # half a step of fp32, relative


def half_step(t):
    return torch.finfo(t).eps / 2


def norm_forward(x, blocks, w_pre, w_post, gate, alpha, beta, eps, offset):
    """(x_out before rounding, size of its terms, 1/rms of the block)."""
    b = sum(t.to(D) for t in blocks)
    rb = (b.square().mean(1, keepdim=True) + eps).rsqrt()
    n = beta * b * rb * (w_post.to(D) + offset)
    if gate is not None:
        n = n * gate.to(D)
    return alpha * x.to(D) + n, (alpha * x.to(D)).abs() + n.abs(), rb


def pre_norm(x_out, w_pre, eps, offset):
    t = x_out.to(D)
    rx = (t.square().mean(1, keepdim=True) + eps).rsqrt()
    return t * rx * (w_pre.to(D) + offset), rx


def norm_backward(dy, dx_out, x, blocks, stats, w_pre, w_post, gate, alpha, beta, offset):
    """({name: gradient}, {name: size of its terms})."""
    rb, rx = stats[0].to(D)[:, None], stats[1].to(D)[:, None]
    dy, xo = dy.to(D), x.to(D)
    wq, wp = w_pre.to(D) + offset, w_post.to(D) + offset
    g = torch.ones(1, dtype=D) if gate is None else gate.to(D)
    xh, bh = xo * rx, sum(t.to(D) for t in blocks) * rb
    u = dy * wq
    ext = torch.zeros_like(xo) if dx_out is None else dx_out.to(D)
    c1, c1a = (u * xh).mean(1, keepdim=True), (u * xh).abs().mean(1, keepdim=True)
    dt = ext + rx * (u - xh * c1)
    dta = ext.abs() + rx * (u.abs() + xh.abs() * c1a)
    z, za = beta * dt * g * wp, abs(beta) * dta * (g * wp).abs()
    db = rb * (z - bh * (z * bh).mean(1, keepdim=True))
    dba = rb * (za + bh.abs() * (za * bh.abs()).mean(1, keepdim=True))
    v, va = beta * dt, abs(beta) * dta
    out = {"dx": alpha * dt, "db": db, "dw_pre": (dy * xh).sum(0), "dw_post": (v * g * bh).sum(0)}
    size = {"dx": abs(alpha) * dta, "db": dba, "dw_pre": (dy * xh).abs().sum(0), "dw_post": (va * (g * bh).abs()).sum(0)}
    if gate is not None:
        dims = 0 if gate.dim() == 1 else 1
        out["dgate"] = (v * bh * wp).sum(dims, keepdim=gate.dim() == 2)
        size["dgate"] = (va * (bh * wp).abs()).sum(dims, keepdim=gate.dim() == 2)
    return out, size


def cdf(u):
    return 0.5 * torch.erfc(-u / math.sqrt(2.0))


def pdf(u):
    return torch.exp(-0.5 * u * u) / math.sqrt(2.0 * math.pi)


def pack(u):
    """(values the codes stand for before scaling, exponent bytes) by search over every e4m3 value."""
    M, F = u.shape
    grid = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(D)
    grid = torch.unique(grid[~grid.isnan()])
    codes, scales = torch.empty(M, F, dtype=D), torch.empty(-(-M // 32), -(-F // 32), dtype=torch.int64)
    for i in range(0, M, 32):
        for j in range(0, F, 32):
            b = u[i:i + 32, j:j + 32].to(D)
            fin = b.isfinite()
            top = float(torch.where(fin, b, 0.0).abs().max())
            e = -117
            while top > 448.0 * 2.0 ** e:
                e += 1
            q = b / 2.0 ** e
            at = torch.bucketize(q, grid).clamp(1, len(grid) - 1)
            lo, hi = grid[at - 1], grid[at]
            near = torch.where((q - lo) < (hi - q), lo, hi)
            tie = (q - lo) == (hi - q)
            # a tie goes to the even code: the one whose position among its sign's values is even
            even = (_code(lo) % 2) == 0
            near = torch.where(tie, torch.where(even, lo, hi), near)
            codes[i:i + 32, j:j + 32] = torch.where(fin, near, float("nan"))
            scales[i // 32, j // 32] = e + 127
    return codes, scales


def _code(v):
    return v.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).to(torch.int64) & 127


def unpack(codes, scales):
    M, F = codes.shape
    s = torch.repeat_interleave(torch.repeat_interleave(scales.to(torch.int32), 32, 0), 32, 1)[:M, :F]
    return torch.ldexp(codes.to(D), s - 127)


def dequantize(codes, scales, zeros, group):
    N, half = codes.shape
    runs = codes.to(torch.int64).view(N, half // 4, 4)
    q = torch.cat([runs & 15, runs >> 4], 2).reshape(N, 2 * half)
    z = torch.full_like(q, 8) if zeros is None else torch.repeat_interleave(zeros.to(torch.int64), group, 1)
    s = torch.repeat_interleave(scales.to(D), group, 1)
    return (q - z).to(D) * s, (q + z).to(D) * s
