"""8-bit Linears and the MLP block of experts in float64 on the CPU, from their
definitions, with the sizes of the terms that each result is summed from."""
import math

import torch

from block_oracle import _code

D = torch.float64
STEP = 2.0 ** -24            # half a step of fp32, relative
BLOCK = 128


def half_step(t):
    return torch.finfo(t).eps / 2


def blocks(n):
    return -(-n // BLOCK)


def width(n):
    return -(-blocks(n) // 4) * 4


def pack(u):
    """(values of the codes, scale bytes [M, width]) of u [M, K] by search over every e4m3 value."""
    M, K = u.shape
    grid = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(D)
    grid = torch.unique(grid[~grid.isnan()])
    codes, scales = torch.empty(M, K, dtype=D), torch.full((M, width(K)), 10, dtype=torch.int64)
    for j in range(0, K, BLOCK):
        b = u[:, j:j + BLOCK].to(D)
        fin = b.isfinite()
        top = torch.where(fin, b, 0.0).abs().amax(1)
        e = torch.full((M,), -117, dtype=torch.int64)
        while (top > 448.0 * torch.exp2(e.to(D))).any():
            e += (top > 448.0 * torch.exp2(e.to(D))).long()
        q = b / torch.exp2(e.to(D))[:, None]
        at = torch.bucketize(torch.where(fin, q, 0.0), grid).clamp(1, len(grid) - 1)
        lo, hi = grid[at - 1], grid[at]
        near = torch.where((q - lo) < (hi - q), lo, hi)
        near = torch.where((q - lo) == (hi - q), torch.where(_code(lo) % 2 == 0, lo, hi), near)
        codes[:, j:j + BLOCK] = torch.where(fin, near, float("nan"))
        scales[:, j // BLOCK] = e + 127
    return codes, scales


def values(codes, scales):
    """Packed rows: what they stand for."""
    each = torch.repeat_interleave(scales.to(torch.int32), BLOCK, 1)[:, :codes.shape[1]]
    return torch.ldexp(codes.to(D), each - 127)


def weight(codes, scales):
    """A weight [N, K] with a scale for each 128 x 128."""
    s = torch.ldexp(torch.ones((), dtype=D), scales.to(torch.int32) - 127) if scales.dtype == torch.uint8 else scales.to(D)
    each = torch.repeat_interleave(torch.repeat_interleave(s, BLOCK, 0), BLOCK, 1)
    return codes.to(D) * each[:codes.shape[0], :codes.shape[1]]


def gelu(y):
    return y * 0.5 * torch.erfc(-y / math.sqrt(2.0))


def columns(M, E=None):
    return blocks(M) * BLOCK if E is None else (M + 127 * min(E, M)) // BLOCK * BLOCK


def order(ids, E):
    """(offsets, src, pos) of ids [T, k], slot by slot."""
    T, k = ids.shape
    lists = [[] for _ in range(E)]
    for slot, e in enumerate(ids.reshape(-1).tolist()):
        if e >= 0:
            lists[e].append(slot)
    offsets, src, pos = [0], [], torch.full((T * k,), -1, dtype=torch.int32)
    for rows in lists:
        for slot in rows:
            pos[slot] = len(src)
            src.append(slot)
        offsets.append(len(src))
    src += [-1] * (T * k - len(src))
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(src, dtype=torch.int32), pos.view(T, k)


def turned(u, offsets=None, src=None, top=0):
    """u [M, K] as the packed transpose's columns lie: [K, Mt]."""
    M, K = u.shape
    if offsets is None:
        out = torch.zeros(K, columns(M), dtype=u.dtype)
        out[:, :M] = u.t()
        return out
    E, R = len(offsets) - 1, M * top if top else M
    out = torch.zeros(K, columns(R, E), dtype=u.dtype)
    col = 0
    for e in range(E):
        for i, r in enumerate(range(offsets[e], offsets[e + 1])):
            out[:, col + i] = u[src[r] // top if top else r]
        col += blocks(int(offsets[e + 1] - offsets[e])) * BLOCK
    return out


def scores(logits, score):
    x = logits.to(D)
    return torch.softmax(x, 1) if score == "softmax" else 1.0 / (1.0 + torch.exp(-x))


def choose(logits, k, score, bias, groups, top_groups, mask):
    """ids [T, k] by sorting (value, number) pairs."""
    T, E = logits.shape
    s = scores(logits, score)
    s = torch.where(torch.isneginf(logits.to(D)), 0.0, s)      # also where a whole row is -inf
    biased = s if bias is None else s + bias.to(D)
    value = logits.to(D) if bias is None else biased
    low = lambda v: float("-inf") if math.isnan(v) else v
    ids = torch.full((T, k), -1, dtype=torch.int32)
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        allowed = range(E)
        if groups > 1:
            n = E // groups
            sums = [(sum(sorted(map(low, biased[t, g * n:(g + 1) * n].tolist()), reverse=True)[:2]), g) for g in range(groups)]
            best = sorted(sums, key=lambda p: (-low(p[0]), p[1]))[:top_groups]
            allowed = [e for _, g in best for e in range(g * n, (g + 1) * n)]
        row = value[t].tolist()
        ids[t] = torch.tensor(sorted(allowed, key=lambda e: (-low(row[e]), e))[:k], dtype=torch.int32)
    return ids


def route_weights(logits, ids, score, renorm, scale):
    s = torch.where(torch.isneginf(logits.to(D)), 0.0, scores(logits, score))
    w = torch.gather(s, 1, ids.clamp(min=0).long())
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0.0, 0.0, w / total)
    return torch.where(ids >= 0, scale * w, 0.0)


def route_gradient(logits, ids, weights, dweights, score, renorm, scale):
    """(gradient, size of its terms), at the weights given."""
    x, g = logits.to(D), dweights.to(D)
    at, routed = ids.clamp(min=0).long(), ids >= 0
    w = torch.where(routed, weights.to(D), 0.0)
    total = (w * g).sum(1, keepdim=True)
    slope = 1.0 if score == "softmax" else 1.0 / (1.0 + torch.exp(torch.gather(x, 1, at)))
    if renorm:
        d = w * (g - total / scale) * slope
        size = w.abs() * (g.abs() + ((w * g).abs().sum(1, keepdim=True) / abs(scale))) * slope
    else:
        d, size = w * g * slope, (w * g * slope).abs()
    out = torch.zeros_like(x).scatter_(1, at, torch.where(routed, d, 0.0))
    big = torch.zeros_like(x).scatter_(1, at, torch.where(routed, size, 0.0))
    if score == "softmax" and not renorm:
        out = torch.where(routed[:, :1], out - torch.softmax(x, 1) * total, 0.0)
        big = big + torch.softmax(x, 1) * (w * g).abs().sum(1, keepdim=True)
    return out, big
