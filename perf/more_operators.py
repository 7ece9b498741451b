"""Measured cases of the 8-bit Linear and of the MLP block of experts.

Five operators: activations packed to e4m3 with one power of two for each 128
values of a row or of a column; tensor-parallel products of such operands
(row-parallel sum over shards, weight gradient); routing of tokens to experts
(scores, bias, groups, top k, weights, the order of the experts' rows, and the
gradient); the experts' products; and the sum of each token's rows, forward and
backward.  ``own`` selects the library's calls; otherwise the operators are
computed by elementary torch operations.
"""
import math

import torch

own = False

BLOCK = 128         # values that share a scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the router of one decode step of 16 tokens: softmax scores, 8 of 64 experts (latency)
        dict(name="route_decode16", op="route", T=16, E=64, k=8, score="softmax", bias=False, groups=1, top_groups=1,
             renorm=True, scale=1.0, masked=False, logits="bf16", backward=False),
        # a training batch: sigmoid scores with a balancing bias, 4 of 8 groups, 8 of 256 experts, and the gradient
        dict(name="route_train16k", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             renorm=True, scale=2.5, masked=True, logits="f32", backward=True),
        # FC1's input of the sequence-parallel block, 8 shards of [2048, 6144], packed for the forward product
        dict(name="pack_rows", op="pack", p=8, M=2048, K=6144, columns=False),
        # an output gradient of the Llama-style layer (4096 tokens), both ways: for dX along rows, for dW down columns
        dict(name="pack_both", op="pack", p=1, M=4096, K=4096, columns=True),
        # one decode step of 16 tokens, row-parallel over 8 shards, weights with fp32 scales
        dict(name="fp8_decode16", op="fp8", p=8, M=16, K=1024, N=8192, wscale="f32", gelu=False, out="bf16"),
        # the Llama-style down projection: 4 shards, 4096 tokens
        dict(name="fp8_down4096", op="fp8", p=4, M=4096, K=4096, N=4096, wscale="u8", gelu=False, out="bf16"),
        # a weight gradient at odd sizes: a ragged batch of 1003 tokens, fp32 result
        dict(name="fp8_dw_odd", op="fp8_dw", p=2, M=1003, R=1360, C=2064, out="f32"),
        # FC1 of 64 experts for 16 tokens with GeLU: each expert's weights are read for two tokens or so
        dict(name="experts_decode16", op="experts", p=1, T=16, E=64, k=8, K=4096, N=1024, skew=0.0, masked=False,
             gather=True, wscale="f32", gelu=True, out="bf16"),
        # FC2 of the same experts for 4096 tokens of a padded batch, uneven loads
        dict(name="experts_prefill4096", op="experts", p=1, T=4096, E=64, k=8, K=1024, N=4096, skew=0.7, masked=True,
             gather=False, wscale="u8", gelu=False, out="bf16"),
        # FC1's weight gradients of 16 experts, two a token, 8192 tokens
        dict(name="experts_dw8192", op="experts_dw", p=1, T=8192, E=16, k=2, R=4096, C=1024, skew=0.7, masked=False,
             out="bf16"),
        # the experts' rows of 4096 tokens summed per token
        dict(name="combine4096", op="combine", T=4096, E=64, k=8, H=4096, skew=0.7, masked=False, backward=False),
        # its backward pass at odd sizes, a padded batch
        dict(name="combine_bwd_odd", op="combine", T=1003, E=60, k=6, H=5000, skew=0.7, masked=True, backward=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, step * int(round(v / step))))


def draw(rng):
    op = rng.choice(["route", "pack", "fp8", "fp8_dw", "experts", "experts_dw", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.choice([2, 3, 8, 15, 20, 32] if groups > 1 else [8, 16, 60, 64, 129, 160, 256, 384])
        top = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(E // groups * top, 16))
        return dict(op=op, T=_log(rng, 1, 16384 * 256 // max(E, 256)), E=E, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top,
                    renorm=rng.random() < 0.7, scale=round(rng.uniform(0.5, 3.0), 2), masked=rng.random() < 0.4,
                    logits=rng.choice(["f32", "bf16"]), backward=rng.random() < 0.5)
    if op == "pack":
        p, K = rng.choice([1, 2, 4, 8]), _log(rng, 64, 16384, 16)
        return dict(op=op, p=p, M=_log(rng, 1, min(8192, (1 << 26) // (K * p))), K=K, columns=rng.random() < 0.5)
    if op == "fp8":
        p = rng.choice([1, 2, 4, 8])
        K = _log(rng, 128, 8192 // p, 16)
        return dict(op=op, p=p, M=_log(rng, 1, 4096), K=K, N=_log(rng, 64, 8192, 8), wscale=rng.choice(["u8", "f32"]),
                    gelu=rng.random() < 0.3, out=rng.choice(["bf16", "f32"]))
    if op == "fp8_dw":
        return dict(op=op, p=rng.choice([1, 2, 4]), M=_log(rng, 1, 4096), R=_log(rng, 64, 4096, 16),
                    C=_log(rng, 64, 4096, 16), out=rng.choice(["f32", "bf16"]))
    E, skew, masked = rng.choice([8, 16, 60, 64]), rng.choice([0.0, 0.5, 1.0]), rng.random() < 0.4
    k = rng.choice([1, 2, 6, 8])
    if op == "experts":
        return dict(op=op, p=rng.choice([1, 1, 2]), T=_log(rng, 1, 4096), E=E, k=k, K=_log(rng, 128, 2048, 16),
                    N=_log(rng, 64, 2048, 8), skew=skew, masked=masked, gather=rng.random() < 0.5,
                    wscale=rng.choice(["u8", "f32"]), gelu=rng.random() < 0.4, out=rng.choice(["bf16", "f32"]))
    if op == "experts_dw":
        return dict(op=op, p=rng.choice([1, 1, 2]), T=_log(rng, 1, 2048), E=E, k=k, R=_log(rng, 64, 1024, 16),
                    C=_log(rng, 64, 1024, 16), skew=skew, masked=masked, out=rng.choice(["f32", "bf16"]))
    H = _log(rng, 64, 8192, 8)
    return dict(op=op, T=_log(rng, 1, min(4096, (1 << 27) // (H * k))), E=E, k=k, H=H, skew=skew, masked=masked,
                backward=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SZ = {"bf16": 2, "f32": 4}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)

    def activations(*shape):
        """Values with a few channels far larger than the others."""
        wide = 1.0 + 7.0 * (torch.rand(shape[-1], device="cuda", generator=g) < 0.02).float()
        return normal(*shape, dtype=torch.float32).mul_(wide).to(torch.bfloat16)

    def weights(*shape):
        """Codes and scales near those of weights N(0, 0.02)."""
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        for part in codes:      # one shard at a time: drawn in 32 bits
            part.copy_(normal(*shape[1:], std=64.0, dtype=torch.float32).clamp_(-448.0, 448.0))
        blocks = shape[:-2] + (-(-shape[-2] // BLOCK), -(-shape[-1] // BLOCK))
        if case["wscale"] == "u8":
            scales = torch.randint(114, 117, blocks, device="cuda", generator=g, dtype=torch.uint8)
        else:
            scales = 0.02 / 64.0 * (0.5 + torch.rand(blocks, device="cuda", generator=g))
        return codes, scales

    def padding(T):
        """A padded batch: the last tokens of each run of 64 are no tokens (None: all are)."""
        if not case["masked"]:
            return None
        lengths = torch.randint(48, 65, (-(-T // 64), 1), device="cuda", generator=g)
        return (torch.arange(64, device="cuda") < lengths).reshape(-1)[:T].contiguous()

    if op == "route":
        T, E = case["T"], case["E"]
        s["x"] = normal(T, E, std=1.5, dtype=_DT[case["logits"]])
        s["bias"] = normal(E, std=0.05, dtype=torch.float32) if case["bias"] else None
        s["mask"] = padding(T)
        s["dweights"] = normal(T, case["k"], dtype=torch.float32) if case["backward"] else None
        return s
    if op == "pack":
        s["u"] = activations(case["p"], case["M"], case["K"])
        return s
    if op == "fp8":
        s["x"] = _pack(activations(case["p"], case["M"], case["K"]))
        s["w"] = weights(case["p"], case["N"], case["K"])
        return s
    if op == "fp8_dw":
        p, M = case["p"], case["M"]
        s["a"] = _pack(_columns(activations(p, M, case["R"])))
        s["b"] = _pack(_columns(normal(p, M, case["C"], std=0.1)))
        return s
    # the order of the experts' rows: k experts a token, popularity falling with the expert's number where skewed
    T, E, k = case["T"], case["E"], case["k"]
    noise = -torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=g).clamp(1e-7, 1.0 - 1e-7)))
    noise -= case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda"))
    ids = torch.sort(noise, dim=1, descending=True).indices[:, :k].to(torch.int32)
    share = torch.rand(T, k, device="cuda", generator=g) + 0.1
    share = share / share.sum(1, keepdim=True)
    mask = padding(T)
    if mask is not None:
        ids = torch.where(mask[:, None], ids, -1)
        share = torch.where(mask[:, None], share, 0.0)
    s["route"] = (ids, share) + _order(ids, E)
    s["bounds"] = [int(v) for v in s["route"][2].tolist()]      # the plain form's copy on the host
    R = T * k
    if op == "experts":
        s["x"] = _pack(activations(case["p"], T if case["gather"] else R, case["K"]))
        s["w"] = weights(case["p"], E, case["N"], case["K"])
        s["w"] = tuple(t.view((case["p"], E) + t.shape[2:]) for t in s["w"])
        return s
    if op == "experts_dw":
        s["a"] = _pack(_columns(activations(case["p"], R, case["R"]), s["route"]))
        s["b"] = _pack(_columns(normal(case["p"], R, case["C"], std=0.1), s["route"]))
        return s
    s["rows"] = normal(R, case["H"])
    s["dy"] = normal(T, case["H"], std=0.1) if case["backward"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from tensor_gemm_reduction_amd import tpfuse as tp
    op = s["op"]
    if op == "route":
        route = tp.expert_route(s["x"], s["k"], score=s["score"], bias=s["bias"], groups=s["groups"],
                                top_groups=s["top_groups"], renorm=s["renorm"], scale=s["scale"], mask=s["mask"])
        out = dict(route._asdict())
        if s["backward"]:
            out["dlogits"] = tp.expert_route_backward(s["dweights"], s["x"], route, score=s["score"],
                                                      renorm=s["renorm"], scale=s["scale"])
        return out
    if op == "pack":
        codes, scales, codes_t, scales_t = tp.fp8_pack(s["u"].unbind(0), columns=s["columns"])
        out = {"codes": codes, "scales": scales}
        if s["columns"]:
            out.update(codes_t=codes_t, scales_t=scales_t)
        return out
    if op == "fp8":
        return {"y": tp.fp8_matmul(s["x"][0].unbind(0), s["x"][1].unbind(0), s["w"][0].unbind(0), s["w"][1].unbind(0),
                                   gelu=s["gelu"], out_dtype=_DT[s["out"]])}
    if op == "fp8_dw":
        return {"dw": tp.fp8_weight_grad(s["a"][0].unbind(0), s["a"][1].unbind(0), s["b"][0].unbind(0),
                                         s["b"][1].unbind(0), out_dtype=_DT[s["out"]])}
    route = tp.ExpertRoute(*s["route"])
    if op == "experts":
        return {"y": tp.expert_matmul(s["x"][0].unbind(0), s["x"][1].unbind(0), s["w"][0].unbind(0),
                                      s["w"][1].unbind(0), route, gather=s["gather"], gelu=s["gelu"],
                                      out_dtype=_DT[s["out"]])}
    if op == "experts_dw":
        return {"dw": tp.expert_weight_grad(s["a"][0].unbind(0), s["a"][1].unbind(0), s["b"][0].unbind(0),
                                            s["b"][1].unbind(0), route, out_dtype=_DT[s["out"]])}
    if s["backward"]:
        drows, dweights = tp.expert_combine_backward(s["dy"], s["rows"], route)
        return {"drows": drows, "dweights": dweights}
    return {"y": tp.expert_combine(s["rows"], route)}


def _run_plain(s):
    op = s["op"]
    if op == "route":
        out = _route(s)
        if s["backward"]:
            out["dlogits"] = _route_backward(s, out["ids"], out["weights"])
        return out
    if op == "pack":
        out = dict(zip(("codes", "scales"), (list(t.unbind(0)) for t in _pack(s["u"]))))
        if s["columns"]:
            out.update(zip(("codes_t", "scales_t"), (list(t.unbind(0)) for t in _pack(_columns(s["u"])))))
        return out
    if op == "fp8":
        y = 0.0
        for k in range(s["p"]):
            y = y + _values(s["x"][0][k], s["x"][1][k]) @ _weight(s["w"][0][k], s["w"][1][k]).t()
        return {"y": (_gelu(y) if s["gelu"] else y).to(_DT[s["out"]])}
    if op == "fp8_dw":
        return {"dw": [(_values(s["a"][0][k], s["a"][1][k]) @ _values(s["b"][0][k], s["b"][1][k]).t()).to(_DT[s["out"]])
                       for k in range(s["p"])]}
    ids, weights, _, src, pos = s["route"]
    at, E = s["bounds"], s["E"]
    if op == "experts":
        y = torch.zeros(src.numel(), s["N"], device="cuda")
        token = (src.long() // s["k"]).clamp(min=0)
        for j in range(s["p"]):
            x = _values(s["x"][0][j], s["x"][1][j])
            for e in range(E):
                if at[e + 1] > at[e]:
                    rows = x[token[at[e]:at[e + 1]]] if s["gather"] else x[at[e]:at[e + 1]]
                    y[at[e]:at[e + 1]] += rows @ _weight(s["w"][0][j, e], s["w"][1][j, e]).t()
        return {"y": (_gelu(y) if s["gelu"] else y).to(_DT[s["out"]])}
    if op == "experts_dw":
        out = []
        for j in range(s["p"]):
            a, b = _values(s["a"][0][j], s["a"][1][j]), _values(s["b"][0][j], s["b"][1][j])
            dw = torch.zeros(E, s["R"], s["C"], dtype=_DT[s["out"]], device="cuda")
            first = 0
            for e in range(E):
                last = first + -(-(at[e + 1] - at[e]) // BLOCK) * BLOCK
                dw[e] = (a[:, first:last] @ b[:, first:last].t()).to(dw.dtype)
                first = last
            out.append(dw)
        return {"dw": out}
    there = (pos >= 0)[:, :, None]
    mine = torch.where(there, s["rows"][pos.clamp(min=0).long()].float(), 0.0)       # [T, k, H]
    if not s["backward"]:
        return {"y": (weights[:, :, None] * mine).sum(1).to(torch.bfloat16)}
    dy = s["dy"].float()
    slot = src.clamp(min=0).long()
    drows = weights.reshape(-1)[slot][:, None] * dy[slot // s["k"]]
    return {"drows": torch.where(src[:, None] >= 0, drows, 0.0).to(torch.bfloat16),
            "dweights": (dy[:, None] * mine).sum(2)}


def _gelu(y):
    return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))


def _blocks(n):
    return -(-n // BLOCK)


def _pack(u):
    """(codes e4m3 [.., K], scale bytes [.., S]): each BLOCK values along the last axis divided by the least power of
    two, from 2^-117 on, that keeps the largest within 448.  S: the blocks rounded up to four, those past K of zeros."""
    K, S = u.shape[-1], -(-_blocks(u.shape[-1]) // 4) * 4
    b = torch.nn.functional.pad(u.float(), (0, S * BLOCK - K)).view(u.shape[:-1] + (S, BLOCK))
    bits = torch.where(torch.isfinite(b), b, 0.0).abs().amax(-1).view(torch.int32)
    scales = (((bits + 0x1FFFFF) >> 23) - 8).clamp(min=10)
    codes = torch.where(torch.isfinite(b), b * torch.exp2((127 - scales).float())[..., None], float("nan"))
    codes = codes.view(u.shape[:-1] + (S * BLOCK,))[..., :K].to(torch.float8_e4m3fn)
    return codes.contiguous(), scales.to(torch.uint8)


def _columns(u, route=None):
    """u [p, M, K] turned to [p, K, Mt]: rows padded with zeros to whole blocks, each expert's by themselves."""
    p, M, K = u.shape
    if route is None:
        return torch.nn.functional.pad(u.transpose(1, 2), (0, -M % BLOCK)).contiguous()
    offsets = route[2].long()
    E = offsets.numel() - 1
    counts = offsets[1:] - offsets[:-1]
    first = torch.cumsum((counts + BLOCK - 1) // BLOCK * BLOCK, 0)
    first = first - (counts + BLOCK - 1) // BLOCK * BLOCK
    out = torch.zeros(p, K, (M + 127 * min(E, M)) // BLOCK * BLOCK, dtype=u.dtype, device=u.device)
    row = torch.arange(M, device=u.device)
    expert = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    routed = row < offsets[E]
    row, expert = row[routed], expert[routed]
    out[:, :, first[expert] + row - offsets[expert]] = u[:, row].transpose(1, 2)
    return out


def _values(codes, scales, dtype=torch.float32):
    """What packed rows stand for."""
    each = torch.repeat_interleave(torch.exp2(scales.to(dtype) - 127.0), BLOCK, -1)[..., :codes.shape[-1]]
    return codes.to(dtype) * each


def _weight(codes, scales, dtype=torch.float32):
    """What a weight [N, K] with a scale for each BLOCK x BLOCK values stands for."""
    s = torch.exp2(scales.to(dtype) - 127.0) if scales.dtype == torch.uint8 else scales.to(dtype)
    s = torch.repeat_interleave(torch.repeat_interleave(s, BLOCK, 0), BLOCK, 1)
    return codes.to(dtype) * s[:codes.shape[0], :codes.shape[1]]


def _route(s):
    """Experts ordered by score + bias in 64 bits (without bias by the logit), the lowest number first among equals."""
    T, E, k = s["T"], s["E"], s["k"]
    x = s["x"].double()
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    biased = score if s["bias"] is None else score + s["bias"].double()
    value = x if s["bias"] is None else biased
    if s["groups"] > 1:
        each = biased.view(T, s["groups"], -1)
        total = torch.sort(each, dim=2, descending=True).values[:, :, :2].sum(2)
        chosen = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        allowed = torch.zeros(T, s["groups"], dtype=torch.bool, device="cuda").scatter_(1, chosen, True)
        value = torch.where(allowed[:, :, None].expand_as(each).reshape(T, E), value, float("-inf"))
    ids = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :k]
    weights = torch.gather(score, 1, ids)
    if s["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    weights = (s["scale"] * weights).float()
    if s["mask"] is not None:
        ids = torch.where(s["mask"][:, None], ids, -1)
        weights = torch.where(s["mask"][:, None], weights, 0.0)
    ids = ids.to(torch.int32)
    offsets, src, pos = _order(ids, E)
    return {"ids": ids, "weights": weights, "offsets": offsets, "src": src, "pos": pos}


def _order(ids, E):
    """(offsets, src, pos): rows sorted by expert, in the order of tokens; slots of no expert have no row."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    counts = (key[None, :] == torch.arange(E, device=ids.device)[:, None]).sum(1)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    row = torch.arange(flat.numel(), device=ids.device)
    pos = torch.empty_like(row)
    pos[order] = row
    src = torch.where(row < offsets[E], order, -1)
    return offsets.to(torch.int32), src.to(torch.int32), torch.where(flat < 0, -1, pos).to(torch.int32).view(ids.shape)


def _route_backward(s, ids, weights):
    x, dw = s["x"].float(), s["dweights"]
    routed = torch.ones_like(ids, dtype=torch.bool) if s["mask"] is None else s["mask"][:, None].expand_as(ids)
    at = ids.clamp(min=0).long()
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    mine = torch.gather(score, 1, at)
    if s["renorm"]:
        da = weights * (dw - (weights * dw).sum(1, keepdim=True) / s["scale"])      # through log score
        d = torch.zeros_like(x).scatter_(1, at, da if s["score"] == "softmax" else da * (1.0 - mine))
    elif s["score"] == "sigmoid":
        d = torch.zeros_like(x).scatter_(1, at, s["scale"] * dw * mine * (1.0 - mine))
    else:
        d = torch.zeros_like(x).scatter_(1, at, s["scale"] * dw)
        d = score * (d - (score * d).sum(1, keepdim=True))
    return torch.where(routed[:, :1], d, 0.0).to(s["x"].dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _width(n):
    return -(-_blocks(n) // 4) * 4


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, sz = case["T"], case["E"], case["k"], _SZ[case["logits"]]
        order = T * k * 16 + (E + 1) * 4
        if not case["backward"]:
            return {"bytes": T * E * sz + order, "flops": T * E * (10 + k)}
        # the gradient reads the logits of the chosen experts alone where the others do not matter
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * E * sz * (3 if dense else 2) + order + T * k * 12, "flops": T * E * (20 + k)}
    if op == "pack":
        p, M, K = case["p"], case["M"], case["K"]
        t = K * (_blocks(M) * BLOCK + _width(M)) if case["columns"] else 0
        return {"bytes": p * (3 * M * K + M * _width(K) + t), "flops": p * M * K * (8 if case["columns"] else 4)}
    if op == "fp8":
        p, M, K, N = case["p"], case["M"], case["K"], case["N"]
        return {"bytes": p * (M * K + M * _blocks(K) + N * K + _blocks(N) * _blocks(K) * (4 if case["wscale"] == "f32" else 1))
                + M * N * _SZ[case["out"]], "flops": 2 * p * M * N * K}
    if op == "fp8_dw":
        p, M, R, C = case["p"], case["M"], case["R"], case["C"]
        return {"bytes": p * ((R + C) * (M + _blocks(M)) + R * C * _SZ[case["out"]]), "flops": 2 * p * M * R * C}
    T, E, k = case["T"], case["E"], case["k"]
    R = T * k * (7 / 8 if case["masked"] else 1)        # rows of tokens, on the average
    # experts that get a token, if all are as popular
    busy = E * (1.0 - (1.0 - k / E) ** T)
    if op == "experts":
        p, K, N = case["p"], case["K"], case["N"]
        rows = min(T, R) if case["gather"] else R
        scale = _blocks(N) * _blocks(K) * (4 if case["wscale"] == "f32" else 1)
        return {"bytes": int(p * (rows * (K + _blocks(K)) + busy * (N * K + scale)) + T * k * (N * _SZ[case["out"]] + 4)),
                "flops": int(2 * p * R * N * K)}
    if op == "experts_dw":
        p, r, c = case["p"], case["R"], case["C"]
        return {"bytes": int(p * ((r + c) * R * (1 + 1 / BLOCK) + E * r * c * _SZ[case["out"]])),
                "flops": int(2 * p * R * r * c)}
    H = case["H"]
    if not case["backward"]:
        return {"bytes": int(R * H * 2 + T * H * 2 + T * k * 8), "flops": int(2 * R * H)}
    return {"bytes": int(T * H * 2 + (R + T * k) * H * 2 + T * k * 16), "flops": int(4 * R * H)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _cdf(u):
    return 0.5 * torch.erfc(-u / math.sqrt(2.0))


def _exact_packed(u, rows):
    """The values that codes stand for before scaling; u's blocks run along the last axis."""
    n = u.shape[-1]
    b = torch.nn.functional.pad(u.to(torch.float64), (0, -n % BLOCK)).unfold(-1, BLOCK, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0)).clamp(min=-117.0)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where((top <= 448.0 * torch.exp2(e - 1)) & (e > -117.0), e - 1, e)
    q = b / torch.exp2(e)
    _, power = torch.frexp(q)
    step = torch.exp2((power - 1).clamp(min=-6).to(torch.float64) - 3.0)
    return (torch.round(q / step) * step).flatten(-2)[..., :n if rows else None]


def _spread(codes, scales):
    """Packed rows in 64 bits, by shifts of the exponent."""
    d = codes.to(torch.float64)
    shift = scales.to(torch.int32) - 127
    for b in range(_blocks(codes.shape[-1])):
        part = d[..., b * BLOCK:(b + 1) * BLOCK]
        part.copy_(torch.ldexp(part, shift[..., b:b + 1]))
    return d


def _spread_weight(codes, scales):
    """A weight in 64 bits, block by block."""
    d = codes.to(torch.float64)
    f = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), scales.to(torch.int32) - 127) \
        if scales.dtype == torch.uint8 else scales.to(torch.float64)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            d[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= f[i, j]
    return d


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op == "route":
        return _exact_route(case, s)
    if op == "pack":
        p = case["p"]
        out = {"codes": [_exact_packed(u, True) for u in s["u"]], "scales": [None] * p}
        if case["columns"]:
            out.update(codes_t=[_exact_packed(u.t(), False) for u in s["u"]], scales_t=[None] * p)
        return out
    if op == "fp8":
        y = torch.zeros(case["M"], case["N"], dtype=d, device="cuda")
        for k in range(case["p"]):
            y.addmm_(_spread(s["x"][0][k], s["x"][1][k]), _spread_weight(s["w"][0][k], s["w"][1][k]).t())
        return {"y": y * _cdf(y) if case["gelu"] else y}
    if op == "fp8_dw":
        return {"dw": [_spread(s["a"][0][k], s["a"][1][k]) @ _spread(s["b"][0][k], s["b"][1][k]).t()
                       for k in range(case["p"])]}
    ids, weights, offsets, src, pos = s["route"]
    E, k = case["E"], case["k"]
    if op == "experts":
        slots = ids.reshape(-1)
        y = torch.zeros(slots.numel(), case["N"], dtype=d, device="cuda")
        for j in range(case["p"]):
            x = _spread(s["x"][0][j], s["x"][1][j])
            for e in range(E):
                mine = torch.nonzero(slots == e)[:, 0]
                if mine.numel():
                    at = pos.reshape(-1)[mine].long()
                    y[at] += x[mine // k if case["gather"] else at] @ _spread_weight(s["w"][0][j, e], s["w"][1][j, e]).t()
        return {"y": y * _cdf(y) if case["gelu"] else y}
    if op == "experts_dw":
        loads = torch.bincount(ids[ids >= 0].long(), minlength=E).tolist()
        out = []
        for j in range(case["p"]):
            a, b = _spread(s["a"][0][j], s["a"][1][j]), _spread(s["b"][0][j], s["b"][1][j])
            dw = torch.zeros(E, case["R"], case["C"], dtype=d, device="cuda")
            col = 0
            for e, n in enumerate(loads):
                dw[e] = a[:, col:col + n] @ b[:, col:col + n].t()
                col += _blocks(n) * BLOCK
            out.append(dw)
        return {"dw": out}
    T, H = case["T"], case["H"]
    if not case["backward"]:
        y = torch.zeros(T, H, dtype=d, device="cuda")
        for j in range(k):
            t = torch.nonzero(pos[:, j] >= 0)[:, 0]
            y[t] += weights[t, j, None].to(d) * s["rows"][pos[t, j].long()].to(d)
        return {"y": y}
    drows = torch.zeros(T * k, H, dtype=d, device="cuda")
    dweights = torch.zeros(T, k, dtype=d, device="cuda")
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        at, dy = pos[t, j].long(), s["dy"][t].to(d)
        drows[at] = weights[t, j, None].to(d) * dy
        dweights[t, j] = torch.linalg.vecdot(dy, s["rows"][at].to(d))
    return {"drows": drows, "dweights": dweights}


def _exact_route(case, s):
    """Weights and the gradient given the choice (whole numbers are compared by themselves)."""
    chosen = _route(s)["ids"]
    x = s["x"].to(torch.float64)
    routed = chosen >= 0
    at = chosen.clamp(min=0).long()
    logit = torch.gather(x, 1, at)
    if case["score"] == "softmax":
        log_score = logit - torch.logsumexp(x, 1, keepdim=True)
        slope = torch.ones_like(logit)
    else:
        log_score = torch.nn.functional.logsigmoid(logit)
        slope = torch.sigmoid(-logit)
    if case["renorm"]:
        weights = case["scale"] * torch.softmax(log_score, 1)
    else:
        weights = case["scale"] * torch.exp(log_score)
    out = {"ids": None, "weights": torch.where(routed, weights, 0.0), "offsets": None, "src": None, "pos": None}
    if case["backward"]:
        # by definition the gradient is taken at the weights in 32 bits
        w = torch.where(routed, weights, 0.0).float().to(torch.float64) if case["renorm"] else weights
        g = w * s["dweights"].to(torch.float64)
        total = g.sum(1, keepdim=True)
        if case["renorm"]:
            d = torch.zeros_like(x).scatter_(1, at, (g - w * total / case["scale"]) * slope)
        elif case["score"] == "sigmoid":
            d = torch.zeros_like(x).scatter_(1, at, g * slope)
        else:
            d = torch.zeros_like(x).scatter_(1, at, g) - torch.softmax(x, 1) * total
        out["dlogits"] = torch.where(routed[:, :1], d, 0.0)
    return out
