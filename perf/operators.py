"""Measured cases of the MLP block's operators around its matrix products.

Three operators of the tensor-parallel MLP block: the norms before and after
it with the block's gate and residual scale (forward and backward), its
activations kept in 8 bits for the backward pass (pack, use in the GeLU's
gradient, use in the weight gradient), and its products with 4-bit weights.
``own`` selects the library's calls; otherwise the operators are computed by
elementary torch operations in 32 bits.
"""
import math

import torch

own = False

BLOCK = 32          # the 8-bit activations share one scale per BLOCK x BLOCK values


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 16 tokens: post-norm, channel gate, residual, next pre-norm (latency)
        _norm("norm_decode16", "norm_fwd", 16, 8192, 1, "bf16", "bf16", "channel", "bf16"),
        # a training batch of the Llama-style layer (4096 tokens, h 4096)
        _norm("norm_train4096", "norm_fwd", 4096, 4096, 1, "bf16", "bf16", "channel", "bf16"),
        # the reduction of four shards' fp32 partials folded in, fp32 residual stream, GPT-3 width
        _norm("norm_partials", "norm_fwd", 2048, 12288, 4, "f32", "f32", "token", "f32"),
        # backward of the sequence-parallel layer (8192 tokens, h 8192)
        _norm("norm_bwd8192", "norm_bwd", 8192, 8192, 1, "bf16", "bf16", "channel", "bf16"),
        # backward at odd sizes, fp32 residual stream, one gate a token, weights stored as offsets from 1
        _norm("norm_bwd_odd", "norm_bwd", 1003, 5000, 1, "f32", "bf16", "token", "f32", offset=True),
        # FC1's output of the Llama-style layer: GeLU and the 8-bit copy in one pass (4 shards)
        dict(name="stash_fwd", op="stash_fwd", p=4, M=4096, F=4096),
        # its use in the backward pass, GPT-3 shapes (8 shards of [2048, 6144])
        dict(name="stash_bwd", op="stash_bwd", p=8, M=2048, F=6144),
        # the down projection's weight gradient from the 8-bit activations (4 shards, fp32 result)
        dict(name="stash_dw4096", op="stash_dw", p=4, M=4096, R=4096, C=4096, out="f32"),
        # the same at odd sizes: a ragged batch of tokens, bf16 result
        dict(name="stash_dw_odd", op="stash_dw", p=2, M=1003, R=1352, C=2056, out="bf16"),
        # one token through one square 4-bit layer (latency)
        dict(name="qweight_one", op="qweight", p=1, M=1, K=8192, N=8192, group=128, zeros=False, gelu=False, out="bf16"),
        # 16 tokens, row-parallel over 8 shards, the smallest groups with zero points
        dict(name="qweight_decode16", op="qweight", p=8, M=16, K=1024, N=8192, group=32, zeros=True, gelu=False, out="bf16"),
        # 64 tokens through the 28672 -> 8192 down projection over 8 shards, fp32 result
        dict(name="qweight_ffn64", op="qweight", p=8, M=64, K=3584, N=8192, group=64, zeros=True, gelu=False, out="f32"),
    ]


def _norm(name, op, M, H, p, x, b, gate, vec, offset=False):
    return dict(name=name, op=op, M=M, H=H, p=p, x=x, b=b, gate=gate, vec=vec, offset=offset,
                alpha=1.0, beta=0.5, eps=1e-6)


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, step * int(round(v / step))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "stash_fwd", "stash_bwd", "stash_dw", "qweight"])
    if op in ("norm_fwd", "norm_bwd"):
        H = _log(rng, 64, 16384, 8)
        p = rng.choice([1, 1, 2, 4])
        M = _log(rng, 1, min(8192, (1 << 26) // (H * p)))
        c = _norm("", op, M, H, p, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]),
                  rng.choice(["none", "channel", "token"]), rng.choice(["bf16", "f32"]), rng.random() < 0.5)
        c["alpha"], c["beta"] = round(rng.uniform(0.5, 1.5), 2), round(rng.uniform(0.1, 1.0), 2)
        del c["name"]
        return c
    if op in ("stash_fwd", "stash_bwd"):
        p, F = rng.choice([1, 2, 4, 8]), _log(rng, 64, 16384, 8)
        return dict(op=op, p=p, M=_log(rng, 1, min(8192, (1 << 26) // (F * p))), F=F)
    if op == "stash_dw":
        return dict(op=op, p=rng.choice([1, 2, 4]), M=_log(rng, 1, 4096), R=_log(rng, 64, 4096, 8),
                    C=_log(rng, 64, 4096, 8), out=rng.choice(["f32", "bf16"]))
    G, p = rng.choice([32, 64, 128]), rng.choice([1, 2, 4, 8])
    K = _log(rng, G, 16384 // p, G)
    return dict(op=op, p=p, M=_log(rng, 1, 64), K=K, N=_log(rng, 16, 16384), group=G, zeros=rng.random() < 0.5,
                gelu=rng.random() < 0.3, out=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SZ = {"bf16": 2, "f32": 4}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype="bf16"):
        return (torch.randn(shape, device="cuda", generator=g) * std).to(_DT[dtype])

    s = dict(case)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        M, H, p, vec = case["M"], case["H"], case["p"], case["vec"]
        base = 0.0 if case["offset"] else 1.0
        s["w_pre"] = (base + 0.2 * torch.randn(H, device="cuda", generator=g)).to(_DT[vec])
        s["w_post"] = (base + 0.2 * torch.randn(H, device="cuda", generator=g)).to(_DT[vec])
        shape = {"none": None, "channel": (H,), "token": (M, 1)}[case["gate"]]
        s["gate"] = None if shape is None else (0.5 + 0.3 * torch.randn(shape, device="cuda", generator=g)).to(_DT[vec])
        s["blocks"] = normal(p, M, H, std=0.7, dtype=case["b"])
        s["x"] = normal(M, H, std=2.0, dtype=case["x"])     # the residual stream (backward: after the block)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(M, H, std=0.5)
            s["dx_out"] = normal(M, H, std=0.5, dtype=case["x"])
            b = s["blocks"].double().sum(0)
            s["stats"] = torch.stack([(t.square().mean(1) + case["eps"]).rsqrt().float()
                                      for t in (b, s["x"].double())])
        return s
    if case["op"] in ("stash_fwd", "stash_bwd", "stash_dw"):
        p, M = case["p"], case["M"]
        F = case["R"] if case["op"] == "stash_dw" else case["F"]
        # pre-activations with a few channels far larger than the others
        wide = 1.0 + 7.0 * (torch.rand(F, device="cuda", generator=g) < 0.02).float()
        u = (torch.randn((p, M, F), device="cuda", generator=g) * wide).to(torch.bfloat16)
        if case["op"] == "stash_fwd":
            s["u"] = u
            return s
        s["codes"], s["scales"] = _pack(u)
        if case["op"] == "stash_bwd":
            s["dh"] = normal(p, M, F, std=0.1)
        else:
            s["dy"] = normal(p, M, case["C"], std=0.1)
        return s
    p, M, K, N, G = case["p"], case["M"], case["K"], case["N"], case["group"]
    s["x"] = normal(p, M, K)
    s["codes"] = torch.randint(0, 256, (p, N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    s["scales"] = (0.002 + 0.008 * torch.rand((p, N, K // G), device="cuda", generator=g)).to(torch.bfloat16)
    s["zeros"] = (torch.randint(5, 12, (p, N, K // G), device="cuda", generator=g, dtype=torch.uint8)
                  if case["zeros"] else None)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from tensor_gemm_reduction_amd import tpfuse as tp
    op = s["op"]
    if op == "norm_fwd":
        x_out, y, stats = tp.block_norm(s["x"], s["blocks"].unbind(0), w_pre=s["w_pre"], w_post=s["w_post"],
                                        gate=s["gate"], alpha=s["alpha"], beta=s["beta"], eps=s["eps"],
                                        unit_offset=s["offset"], want_stats=True)
        return {"x_out": x_out, "y": y, "stats": stats}
    if op == "norm_bwd":
        dx, db, dw_pre, dw_post, dgate = tp.block_norm_backward(
            s["dy"], s["dx_out"], s["x"], s["blocks"].unbind(0), s["stats"], w_pre=s["w_pre"], w_post=s["w_post"],
            gate=s["gate"], alpha=s["alpha"], beta=s["beta"], unit_offset=s["offset"])
        return {"dx": dx, "db": db, "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}
    if op == "stash_fwd":
        h, codes, scales = tp.stash_pack(s["u"].unbind(0), gelu=True)
        return {"h": h, "codes": codes, "scales": scales}
    if op == "stash_bwd":
        du, h = tp.stash_backward(s["codes"].unbind(0), s["scales"].unbind(0), s["dh"].unbind(0))
        return {"du": du, "h": h}
    if op == "stash_dw":
        return {"dw": tp.stash_weight_grad(s["codes"].unbind(0), s["scales"].unbind(0), s["dy"].unbind(0),
                                           out_dtype=_DT[s["out"]])}
    zeros = None if s["zeros"] is None else s["zeros"].unbind(0)
    return {"y": tp.qweight_matmul(s["x"].unbind(0), s["codes"].unbind(0), s["scales"].unbind(0), zeros,
                                   group=s["group"], gelu=s["gelu"], out_dtype=_DT[s["out"]])}


def _run_plain(s):
    op = s["op"]
    if op == "norm_fwd":
        off = 1.0 if s["offset"] else 0.0
        b = s["blocks"].float().sum(0)
        rb = 1.0 / torch.sqrt(b.square().mean(1, keepdim=True) + s["eps"])
        n = s["beta"] * (b * rb * (s["w_post"].float() + off))
        if s["gate"] is not None:
            n = n * s["gate"].float()
        x_out = (s["alpha"] * s["x"].float() + n).to(s["x"].dtype)
        t = x_out.float()       # the next norm sees the residual stream as it is stored
        rx = 1.0 / torch.sqrt(t.square().mean(1, keepdim=True) + s["eps"])
        y = (t * rx * (s["w_pre"].float() + off)).to(torch.bfloat16)
        return {"x_out": x_out, "y": y, "stats": torch.stack([rb[:, 0], rx[:, 0]])}
    if op == "norm_bwd":
        off = 1.0 if s["offset"] else 0.0
        rb, rx = s["stats"][0][:, None], s["stats"][1][:, None]
        xh = s["x"].float() * rx
        dy = s["dy"].float()
        u = dy * (s["w_pre"].float() + off)
        dt = s["dx_out"].float() + rx * (u - xh * (u * xh).mean(1, keepdim=True))
        bh = s["blocks"].float().sum(0) * rb
        gate = 1.0 if s["gate"] is None else s["gate"].float()
        v = s["beta"] * dt
        z = v * gate * (s["w_post"].float() + off)
        db = rb * (z - bh * (z * bh).mean(1, keepdim=True))
        n = v * bh * (s["w_post"].float() + off)
        dgate = None if s["gate"] is None else n.sum(0) if s["gate"].dim() == 1 else n.sum(1, keepdim=True)
        return {"dx": (s["alpha"] * dt).to(s["x"].dtype), "db": db.to(torch.bfloat16),
                "dw_pre": (dy * xh).sum(0), "dw_post": (v * gate * bh).sum(0), "dgate": dgate}
    if op == "stash_fwd":
        u = s["u"].float()
        h = (0.5 * u * (1.0 + torch.erf(u * math.sqrt(0.5)))).to(torch.bfloat16)
        codes, scales = _pack(s["u"])
        return {"h": list(h.unbind(0)), "codes": list(codes.unbind(0)), "scales": list(scales.unbind(0))}
    if op == "stash_bwd":
        u = _unpack(s["codes"], s["scales"], torch.float32)
        phi = 0.5 * (1.0 + torch.erf(u * math.sqrt(0.5)))
        du = s["dh"].float() * (phi + u * torch.exp(-0.5 * u * u) * (1.0 / math.sqrt(2.0 * math.pi)))
        return {"du": list(du.to(torch.bfloat16).unbind(0)), "h": list((u * phi).to(torch.bfloat16).unbind(0))}
    if op == "stash_dw":
        u = _unpack(s["codes"], s["scales"], torch.float32)
        dw = torch.matmul(u.transpose(1, 2).contiguous(), s["dy"].float())
        return {"dw": list(dw.to(_DT[s["out"]]).unbind(0))}
    w = _dequantize(s, torch.float32)
    M = s["x"].shape[1]
    y = s["x"].float().permute(1, 0, 2).reshape(M, -1) @ w.permute(1, 0, 2).reshape(w.shape[1], -1).t()
    if s["gelu"]:
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return {"y": y.to(_DT[s["out"]])}


def _pad(t):
    """[p, M, F] padded with zeros to whole blocks, as [p, M/B, B, F/B, B]."""
    p, M, F = t.shape
    t = torch.nn.functional.pad(t, (0, -F % BLOCK, 0, -M % BLOCK))
    return t.reshape(p, t.shape[1] // BLOCK, BLOCK, t.shape[2] // BLOCK, BLOCK)


def _pack(u):
    """(codes e4m3, scale bytes): each 32 x 32 block divided by a power of two that brings its largest value to (224, 448]."""
    b = _pad(u.float())
    bits = torch.where(torch.isfinite(b), b, 0.0).abs().amax(dim=(2, 4)).view(torch.int32)
    scales = (((bits + 0x1FFFFF) >> 23) - 8).clamp(min=10)
    inv = torch.exp2((127 - scales).float())
    codes = torch.where(torch.isfinite(b), b * inv[:, :, None, :, None], float("nan"))
    p, mb, _, fb, _ = b.shape
    codes = codes.reshape(p, mb * BLOCK, fb * BLOCK)[:, :u.shape[1], :u.shape[2]].contiguous()
    return codes.to(torch.float8_e4m3fn), scales.to(torch.uint8)


def _unpack(codes, scales, dtype):
    b = _pad(codes.to(dtype)) * torch.exp2(scales.to(dtype) - 127.0)[:, :, None, :, None]
    p, mb, _, fb, _ = b.shape
    return b.reshape(p, mb * BLOCK, fb * BLOCK)[:, :codes.shape[1], :codes.shape[2]]


def _dequantize(s, dtype):
    """The weights [p, N, K]: byte j of each 4 holds code j (low half) and code j + 4 (high half)."""
    p, N, half = s["codes"].shape
    four = s["codes"].view(p, N, half // 4, 4)
    q = torch.cat([four & 15, four >> 4], dim=3).view(p, N, -1, s["group"]).to(dtype)
    z = 8.0 if s["zeros"] is None else s["zeros"].to(dtype)[..., None]
    return ((q - z) * s["scales"].to(dtype)[..., None]).view(p, N, 2 * half)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        M, H, p, sx, sb, sv = case["M"], case["H"], case["p"], _SZ[case["x"]], _SZ[case["b"]], _SZ[case["vec"]]
        gate = {"none": 0, "channel": H, "token": M}[case["gate"]]
        if op == "norm_fwd":
            return {"bytes": M * H * (sx + p * sb + sx + 2) + (2 * H + gate) * sv + 8 * M, "flops": M * H * (p + 10)}
        return {"bytes": M * H * (2 + 3 * sx + p * sb + 2) + (2 * H + gate) * (sv + 4) + 8 * M,
                "flops": M * H * (p + 30)}
    if op in ("stash_fwd", "stash_bwd"):
        n, blocks = case["p"] * case["M"] * case["F"], case["p"] * -(-case["M"] // BLOCK) * -(-case["F"] // BLOCK)
        return {"bytes": n * (5 if op == "stash_fwd" else 7) + blocks, "flops": n * 25}
    if op == "stash_dw":
        p, M, R, C = case["p"], case["M"], case["R"], case["C"]
        return {"bytes": p * (M * R + M * C * 2 + R * C * _SZ[case["out"]] + -(-M // BLOCK) * -(-R // BLOCK)),
                "flops": 2 * p * M * R * C}
    p, M, K, N = case["p"], case["M"], case["K"], case["N"]
    groups = p * N * (K // case["group"])
    return {"bytes": p * N * K // 2 + groups * (3 if case["zeros"] else 2) + p * M * K * 2 + M * N * _SZ[case["out"]],
            "flops": 2 * p * M * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _normal_cdf(u):
    return 0.5 * torch.erfc(-u / math.sqrt(2.0))


def _spread(scales, M, F):
    """A block's scale for each of its values: [p, M, F]."""
    each = torch.repeat_interleave(torch.repeat_interleave(scales, BLOCK, 1), BLOCK, 2)
    return each[:, :M, :F]


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op == "norm_fwd":
        H, off = case["H"], float(case["offset"])
        b = torch.zeros(case["M"], H, dtype=d, device="cuda")
        for part in s["blocks"]:
            b += part.to(d)
        rb = (torch.linalg.vector_norm(b, dim=1) ** 2 / H + case["eps"]) ** -0.5
        gate = torch.ones(1, dtype=d, device="cuda") if s["gate"] is None else s["gate"].to(d)
        post = torch.einsum("mh,m,h->mh", b, rb, s["w_post"].to(d) + off) * gate
        x_out = case["alpha"] * s["x"].to(d) + case["beta"] * post
        kept = x_out.to(s["x"].dtype).to(d)     # by definition the next norm is of the stored residual stream
        rx = (torch.linalg.vector_norm(kept, dim=1) ** 2 / H + case["eps"]) ** -0.5
        return {"x_out": x_out, "y": torch.einsum("mh,m,h->mh", kept, rx, s["w_pre"].to(d) + off),
                "stats": torch.stack([rb, rx])}
    if op == "norm_bwd":
        # the vector-Jacobian product of t = x (held), y = t rx w and of x_out = alpha x + beta gate n(b), with the
        # projections written as inner products along a row
        off, H = float(case["offset"]), case["H"]
        rb, rx = s["stats"].to(d)
        t, dy = s["x"].to(d), s["dy"].to(d)
        wy = dy * (s["w_pre"].to(d) + off)
        along = torch.linalg.vecdot(wy, t) * rx ** 3 / H
        dt = s["dx_out"].to(d) + wy * rx[:, None] - t * along[:, None]
        b = torch.zeros_like(t)
        for part in s["blocks"]:
            b += part.to(d)
        gate = torch.ones(1, dtype=d, device="cuda") if s["gate"] is None else s["gate"].to(d)
        w = s["w_post"].to(d) + off
        bar = case["beta"] * dt
        dn = bar * gate * w
        db = dn * rb[:, None] - b * (torch.linalg.vecdot(dn, b) * rb ** 3 / H)[:, None]
        dgate = None
        if s["gate"] is not None:
            dgate = (rb @ (bar * b)) * w if s["gate"].dim() == 1 else (((bar * b) @ w) * rb)[:, None]
        return {"dx": case["alpha"] * dt, "db": db, "dw_pre": rx @ (dy * t), "dw_post": rb @ (bar * gate * b),
                "dgate": dgate}
    if op == "stash_fwd":
        u = s["u"].to(d)
        p, M, F = u.shape
        top = torch.nn.functional.pad(u.abs(), (0, -F % BLOCK, 0, -M % BLOCK))
        top = top.unfold(1, BLOCK, BLOCK).unfold(2, BLOCK, BLOCK).amax(dim=(3, 4))
        # the least power of two that keeps the block's largest value within 448, and not below 2^-117
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0)).clamp(min=-117.0)
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
        e = torch.where((top <= 448.0 * torch.exp2(e - 1)) & (e > -117.0), e - 1, e)
        q = u / torch.exp2(_spread(e, M, F))
        _, power = torch.frexp(q)
        step = torch.exp2((power - 1).clamp(min=-6).to(d) - 3.0)
        return {"h": list((u * _normal_cdf(u)).unbind(0)), "codes": list((torch.round(q / step) * step).unbind(0)),
                "scales": [None] * p}
    if op == "stash_bwd":
        p, M, F = s["codes"].shape
        u = torch.ldexp(s["codes"].to(d), _spread(s["scales"], M, F).to(torch.int32) - 127)
        density = torch.exp(u.square() / -2.0) / math.sqrt(2.0 * math.pi)
        cdf = _normal_cdf(u)
        return {"du": list((s["dh"].to(d) * torch.addcmul(cdf, u, density)).unbind(0)), "h": list((u * cdf).unbind(0))}
    if op == "stash_dw":
        p, M, R = s["codes"].shape
        u = torch.ldexp(s["codes"].to(d), _spread(s["scales"], M, R).to(torch.int32) - 127)
        return {"dw": [u[k].t() @ s["dy"][k].to(d) for k in range(p)]}
    G, N = case["group"], case["N"]
    y = torch.zeros(case["M"], N, dtype=d, device="cuda")
    shift = torch.tensor([0, 0, 0, 0, 4, 4, 4, 4], device="cuda", dtype=torch.uint8)
    for k in range(case["p"]):
        # code i of a run of 8 is in byte i % 4, its low half for i < 4
        runs = s["codes"][k].view(N, -1, 1, 4).expand(-1, -1, 2, -1).reshape(N, -1, 8)
        q = ((runs >> shift) % 16).reshape(N, -1).to(d)
        zero = 8.0 if s["zeros"] is None else torch.repeat_interleave(s["zeros"][k], G, 1).to(d)
        w = (q - zero) * torch.repeat_interleave(s["scales"][k], G, 1).to(d)
        y += s["x"][k].to(d) @ w.t()
    return {"y": y * _normal_cdf(y) if case["gelu"] else y}
