"""GPU parity of the MLP block's operators (norms, 8-bit activations, 4-bit
weight products) with float64 on the CPU.

Tolerances count roundings: half a step of the output's type relative to the
result, and a multiple of 2^-24 of the sum of the magnitudes that an fp32 sum
runs over.  Every operand sits between NaNs, so that a value read from outside
it shows."""
import pytest
import torch

import block_oracle as O
from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
D = torch.float64


def framed(t):
    """A copy of `t` on the GPU with 256 bytes of NaN (0xff) on both sides."""
    if t is None:
        return None
    n = t.numel() * t.element_size()
    buf = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    v = buf[256:256 + n].view(t.dtype).view(t.shape)
    v.copy_(t)
    return v


def frame(ts):
    return [framed(t) for t in ts]


def rand(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def close(got, want, bound, what):
    got = got.detach().cpu().to(D)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out, worst excess " \
                          f"{float(((got - want).abs() - bound)[bad].max()):.3e}"


NORMS = [  # M, H, p, x, blocks, gate, vectors, offset
    (1, 8, 1, BF, BF, None, BF, False),
    (7, 64, 2, F32, BF, "channel", F32, True),
    (5, 520, 1, BF, F32, "token", BF, False),
    (3, 1032, 3, BF, BF, "channel", F32, False),
    (2, 2048, 8, F32, F32, None, F32, True),
    (33, 4104, 4, BF, F32, "token", F32, True),
    (600, 5000, 1, F32, BF, "token", F32, True),
    (1030, 264, 2, BF, BF, "channel", BF, False),
    (5, 8200, 2, BF, BF, "channel", BF, False),
    (3, 16384, 4, F32, F32, "token", BF, False),
    (2, 32768, 16, BF, BF, "channel", BF, True),
]


def norm_case(M, H, p, xt, bt, gate, vt, offset, seed=0):
    g = torch.Generator().manual_seed(seed + M * 131 + H)
    base = 0.0 if offset else 1.0
    c = dict(x=rand(g, M, H, std=2.0, dtype=xt), blocks=[rand(g, M, H, std=0.7, dtype=bt) for _ in range(p)],
             w_pre=(base + rand(g, H, std=0.2, dtype=F32)).to(vt), w_post=(base + rand(g, H, std=0.2, dtype=F32)).to(vt),
             gate=None if gate is None else (0.5 + rand(g, *((H,) if gate == "channel" else (M, 1)), std=0.3,
                                                        dtype=F32)).to(vt),
             dy=rand(g, M, H, std=0.5), dx_out=rand(g, M, H, std=0.5, dtype=xt))
    if M > 2:                    # a block that put out nothing for a token, and a closed gate
        for b in c["blocks"]:
            b[1] = 0
        if gate == "token":
            c["gate"][2] = 0
    return c


# Statistics: a row's sum of squares is added by threads of at most 32 values,
# a wave's 6 exchanges and 16 waves, so at most 54 roundings; with the products,
# the mean, the root and the factors after it 64 covers them.
ROUNDINGS = 64 * O.STEP


@pytest.mark.parametrize("M,H,p,xt,bt,gate,vt,offset", NORMS)
def test_block_norm(M, H, p, xt, bt, gate, vt, offset):
    c = norm_case(M, H, p, xt, bt, gate, vt, offset)
    alpha, beta, eps, off = 0.9, 0.7, 1e-6, float(offset)
    x, blocks = framed(c["x"]), frame(c["blocks"])
    kw = dict(w_pre=framed(c["w_pre"]), w_post=framed(c["w_post"]), gate=framed(c["gate"]), alpha=alpha, beta=beta,
              eps=eps, unit_offset=offset)
    x_out, y, stats = tp.block_norm(x, blocks, want_stats=True, **kw)
    want, size, rb = O.norm_forward(c["x"], c["blocks"], c["w_pre"], c["w_post"], c["gate"], alpha, beta, eps, off)
    acc = (ROUNDINGS + p * O.STEP) * size + p * O.STEP * abs(beta) * _block_size(c, rb, off)
    close(x_out, want, acc + (O.half_step(xt) * want.abs() if xt is BF else O.STEP * want.abs()), "x_out")
    wy, rx = O.pre_norm(x_out.cpu(), c["w_pre"], eps, off)
    close(y, wy, (O.half_step(BF) + ROUNDINGS) * wy.abs(), "y")
    close(stats[1], rx[:, 0], ROUNDINGS * rx[:, 0], "1/rms of x_out")
    # the block's own sum may cancel: its terms' roundings against its root mean square
    spread = sum(b.to(D).abs() for b in c["blocks"]).square().mean(1).sqrt() * rb[:, 0]
    close(stats[0], rb[:, 0], (ROUNDINGS + p * O.STEP * spread) * rb[:, 0], "1/rms of the block")
    # in place, without statistics, the same bits
    x2 = x.clone()
    got = tp.block_norm(x2, blocks, x_out=x2, **kw)
    assert got[0] is x2 and got[2] is None
    assert torch.equal(x2, x_out) and torch.equal(got[1], y)


def _block_size(c, rb, off):
    s = sum(b.to(D).abs() for b in c["blocks"])
    n = s * rb * (1 + s.square().mean(1, keepdim=True).sqrt() * rb) * (c["w_post"].to(D) + off).abs()
    return n if c["gate"] is None else n * c["gate"].to(D).abs()


@pytest.mark.parametrize("M,H,p,xt,bt,gate,vt,offset", NORMS)
def test_block_norm_backward(M, H, p, xt, bt, gate, vt, offset):
    c = norm_case(M, H, p, xt, bt, gate, vt, offset, seed=1)
    alpha, beta, off = 1.1, 0.6, float(offset)
    _, _, rb = O.norm_forward(c["x"], c["blocks"], c["w_pre"], c["w_post"], c["gate"], 1, 1, 1e-6, off)
    _, rx = O.pre_norm(c["x"], c["w_pre"], 1e-6, off)
    stats = torch.stack([rb[:, 0], rx[:, 0]]).float()
    for dx_out in (c["dx_out"], None):
        want, size = O.norm_backward(c["dy"], dx_out, c["x"], c["blocks"], stats, c["w_pre"], c["w_post"], c["gate"],
                                     alpha, beta, off)
        args = (framed(c["dy"]), framed(dx_out), framed(c["x"]), frame(c["blocks"]), framed(stats))
        kw = dict(w_pre=framed(c["w_pre"]), w_post=framed(c["w_post"]), gate=framed(c["gate"]), alpha=alpha, beta=beta,
                  unit_offset=offset)
        got = dict(zip(("dx", "db", "dw_pre", "dw_post", "dgate"), tp.block_norm_backward(*args, **kw)))
        assert (got["dgate"] is None) == (gate is None)
        # what the shards' sum rounds off, against the sum itself (it may cancel)
        mag = sum(b.to(D).abs() for b in c["blocks"])
        ratio = float((mag.square().mean(1).sqrt() * stats[0].to(D)).max())
        for name, w in want.items():
            rows = M if name in ("dw_pre", "dw_post") or (name == "dgate" and gate == "channel") else 0
            # a column's sum: ceil(M / groups) rows in a register, then 16 strips of groups
            bound = (2 * ROUNDINGS + min(rows, 64) * O.STEP + p * O.STEP * (1 + ratio)) * size[name]
            if p > 1 and name != "dx":
                bound = bound + p * O.STEP * _cancel(name, c, stats, beta, off, size, mag)
            t = got[name].dtype
            close(got[name], w, bound + (O.half_step(t) if t is BF else O.STEP) * w.abs(), name)
        again = tp.block_norm_backward(*args, **kw)
        for a, b in zip(again, got.values()):
            assert a is None or torch.equal(a, b)


def _cancel(name, c, stats, beta, off, size, mag):
    """Size of each result with every shard's magnitude in place of the sum."""
    if name == "dw_pre":
        return torch.zeros_like(size[name])
    g = torch.ones(1, dtype=D) if c["gate"] is None else c["gate"].to(D).abs()
    wp = (c["w_post"].to(D) + off).abs()
    bh = mag * stats[0].to(D)[:, None]
    dt = size["dx"] / 1.1
    if name == "db":
        z = beta * dt * g * wp
        return stats[0].to(D)[:, None] * bh * (z * bh).mean(1, keepdim=True) * 2
    if name == "dw_post":
        return (beta * dt * g * bh).sum(0)
    dims = 0 if c["gate"].dim() == 1 else 1
    return (beta * dt * bh * wp).sum(dims, keepdim=c["gate"].dim() == 2)


def activations(g, M, F, special=True):
    u = rand(g, M, F) * (1 + 7 * (torch.rand(F, generator=g) < 0.05)).to(BF)
    if special and M * F >= 64:
        flat = u.view(-1)
        vals = [float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 3.3e38, 1e-39, -1e-40, 1e-30]
        flat[torch.randperm(flat.numel(), generator=g)[:len(vals)]] = torch.tensor(vals).to(BF)
        if M > 32 and F > 64:
            u[32:64, 32:64] = 0                       # a block of zeros
            u[:32, :32] = rand(g, 32, 32, std=1e-38)  # one below the smallest factor
    return u


STASHES = [(1, 8, 1), (1, 64, 2), (31, 40, 1), (33, 200, 2), (64, 128, 4), (100, 264, 1), (65, 1352, 3), (40, 2056, 16)]


@pytest.mark.parametrize("M,F,p", STASHES)
@pytest.mark.parametrize("gelu", [True, False])
def test_stash_pack(M, F, p, gelu):
    g = torch.Generator().manual_seed(M + F)
    us = [activations(g, M, F) for _ in range(p)]
    h, codes, scales = tp.stash_pack(frame(us), gelu=gelu)
    assert (h is None) == (not gelu)
    for k, u in enumerate(us):
        want, byte = O.pack(u)
        assert torch.equal(scales[k].cpu().to(torch.int64), byte)
        got = codes[k].cpu().to(F32).to(D)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
        if gelu:
            check_gelu(h[k], u.to(D), "h")


def check_gelu(h, u, what):
    want = u * O.cdf(u)
    got = h.cpu().to(D)
    fin = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~fin].nan_to_num(), want[~fin].nan_to_num())
    # the fit (5e-6), the exponent's argument (u^2 / 2 2^-23, below 1e-5 while the result is not
    # subnormal), then half a step; subnormal results may be flushed
    close(got[fin], want[fin], (O.half_step(BF) + 2.0 ** -15) * want[fin].abs() + 2.0 ** -126, what)


@pytest.mark.parametrize("M,F,p", STASHES)
def test_stash_backward(M, F, p):
    g = torch.Generator().manual_seed(M * 3 + F)
    us = [activations(g, M, F, special=False) * 2 for _ in range(p)]
    _, codes, scales = tp.stash_pack([u.cuda() for u in us], gelu=False)
    dh = [rand(g, M, F, std=0.1) for _ in range(p)]
    codes8 = [c.cpu().view(torch.uint8) for c in codes]
    if M * F >= 64:
        codes8[0].view(-1)[5] = 0x7f       # a value that was not finite
    du, h = tp.stash_backward([framed(c).view(torch.float8_e4m3fn) for c in codes8], frame([s.cpu() for s in scales]),
                              frame(dh))
    for k in range(p):
        u = O.unpack(codes8[k].view(torch.float8_e4m3fn).to(F32), scales[k].cpu())
        check_gelu(h[k], u, "h")
        d = dh[k].to(D)
        want, size = d * (O.cdf(u) + u * O.pdf(u)), d.abs() * (O.cdf(u) + u.abs() * O.pdf(u))
        fin = want.isfinite()
        assert torch.equal(du[k].cpu().isnan(), want.isnan())
        close(du[k].cpu()[fin], want[fin], O.half_step(BF) * want[fin].abs() + 2.0 ** -15 * size[fin] + 2.0 ** -126, "du")


GRADS = [  # p, M, R, C
    (1, 1, 8, 8), (2, 31, 64, 136), (1, 32, 256, 256), (2, 33, 264, 520), (1, 63, 72, 1024), (1, 64, 512, 264),
    (3, 65, 136, 72), (1, 200, 1352, 264), (2, 1003, 328, 600), (1, 4100, 64, 64), (16, 40, 40, 56), (1, 700, 2048, 64),
    (4, 513, 1024, 1024),
]


@pytest.mark.parametrize("p,M,R,C", GRADS)
@pytest.mark.parametrize("out", [F32, BF])
def test_stash_weight_grad(p, M, R, C, out):
    g = torch.Generator().manual_seed(M + R + C)
    us = [activations(g, M, R, special=False) for _ in range(p)]
    _, codes, scales = tp.stash_pack([u.cuda() for u in us], gelu=False)
    dy = [rand(g, M, C, std=0.1) for _ in range(p)]
    cf = [framed(c.cpu().view(torch.uint8)).view(torch.float8_e4m3fn) for c in codes]
    sf, yf = frame([s.cpu() for s in scales]), frame(dy)
    dw = tp.stash_weight_grad(cf, sf, yf, out_dtype=out)
    for k in range(p):
        u, y = O.unpack(codes[k].cpu().to(F32), scales[k].cpu()), dy[k].to(D)
        want, size = u.t() @ y, u.abs().t() @ y.abs()
        close(dw[k], want, (M + 8) * O.STEP * size + (O.half_step(BF) * want.abs() if out is BF else 0), f"dw[{k}]")
    again = tp.stash_weight_grad(cf, sf, yf, out_dtype=out)
    assert all(torch.equal(a, b) for a, b in zip(again, dw))


def test_stash_weight_grad_whole_numbers():
    """Small whole numbers in both operands: every sum is exact, in any order."""
    g = torch.Generator().manual_seed(3)
    for p, M, R, C in ((1, 95, 320, 136), (2, 300, 520, 264)):
        u = [torch.randint(-4, 5, (M, R), generator=g).to(BF) for _ in range(p)]
        y = [torch.randint(-3, 4, (M, C), generator=g).to(BF) for _ in range(p)]
        _, codes, scales = tp.stash_pack([t.cuda() for t in u], gelu=False)
        dw = tp.stash_weight_grad(codes, scales, [t.cuda() for t in y])
        for k in range(p):
            assert torch.equal(dw[k].cpu().to(D), u[k].to(D).t() @ y[k].to(D))


QWEIGHTS = [  # p, M, K, N, group, zeros, gelu
    (1, 1, 32, 1, 32, False, False), (1, 1, 128, 16, 128, True, False), (2, 3, 96, 17, 32, True, False),
    (1, 16, 192, 100, 64, False, True), (8, 16, 256, 333, 32, True, False), (1, 17, 640, 64, 128, True, True),
    (4, 31, 320, 50, 64, True, False), (1, 33, 1024, 129, 128, False, False), (3, 64, 416, 260, 32, True, False),
    (1, 65, 384, 48, 128, True, False), (2, 130, 160, 33, 32, False, True), (16, 2, 64, 24, 64, True, False),
    (1, 1, 8192, 272, 128, False, False), (1, 40, 4000, 520, 32, True, False), (1, 5, 14336, 16, 128, True, False),
]


def qweight_case(p, M, K, N, group, zeros, seed=0):
    g = torch.Generator().manual_seed(seed + M + K + N)
    nz = (N, K // group)
    return dict(x=[rand(g, M, K) for _ in range(p)],
                codes=[torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8) for _ in range(p)],
                scales=[(0.002 + 0.008 * torch.rand(nz, generator=g)).to(BF) for _ in range(p)],
                zeros=[torch.randint(0, 16, nz, generator=g, dtype=torch.uint8) for _ in range(p)] if zeros else None)


@pytest.mark.parametrize("p,M,K,N,group,zeros,gelu", QWEIGHTS)
@pytest.mark.parametrize("out", [F32, BF])
def test_qweight_matmul(p, M, K, N, group, zeros, gelu, out):
    c = qweight_case(p, M, K, N, group, zeros)
    args = (frame(c["x"]), frame(c["codes"]), frame(c["scales"]), frame(c["zeros"]) if zeros else None)
    kw = dict(group=group, gelu=gelu, out_dtype=out)
    y = tp.qweight_matmul(*args, **kw)
    want, size = torch.zeros(M, N, dtype=D), torch.zeros(M, N, dtype=D)
    for k in range(p):
        w, wa = O.dequantize(c["codes"][k], c["scales"][k], c["zeros"][k] if zeros else None, group)
        want += c["x"][k].to(D) @ w.t()
        size += c["x"][k].to(D).abs() @ wa.t()
    # a group's sums round once a product at most, the joining once a group
    bound = (group + p * K / group + 16) * O.STEP * size
    if gelu:
        bound = 1.13 * bound + 2.0 ** -20 * want.abs()     # |GeLU'| < 1.13; erf's own error
        want = want * O.cdf(want)
    close(y, want, bound + (O.half_step(BF) * want.abs() if out is BF else 0), "y")
    assert torch.equal(tp.qweight_matmul(*args, **kw), y)


def test_qweight_whole_numbers():
    """Whole numbers with a power of two for a scale: exact in any order."""
    g = torch.Generator().manual_seed(9)
    for p, M, K, N, group in ((1, 4, 256, 40, 32), (2, 20, 128, 64, 64), (1, 64, 384, 200, 128)):
        c = qweight_case(p, M, K, N, group, True)
        x = [torch.randint(-8, 9, (M, K), generator=g).to(BF) for _ in range(p)]
        s = [torch.full((N, K // group), 0.25).to(BF) for _ in range(p)]
        y = tp.qweight_matmul(frame(x), frame(c["codes"]), frame(s), frame(c["zeros"]), group=group, out_dtype=F32)
        want = sum(x[k].to(D) @ O.dequantize(c["codes"][k], s[k], c["zeros"][k], group)[0].t() for k in range(p))
        assert torch.equal(y.cpu().to(D), want)


def test_side_stream_and_graph():
    """Calls on another stream, and replays of a captured graph with new inputs, give the eager bits."""
    M, H, p = 48, 1024, 2
    c = norm_case(M, H, p, BF, F32, "channel", F32, False)
    q = qweight_case(p, M, H, 512, 64, True)
    x, blocks, wq, wp = c["x"].cuda(), [b.cuda() for b in c["blocks"]], c["w_pre"].cuda(), c["w_post"].cuda()
    gate, dy, dxo = c["gate"].cuda(), c["dy"].cuda(), c["dx_out"].cuda()
    codes, scales, zeros = ([t.cuda() for t in q[n]] for n in ("codes", "scales", "zeros"))

    def step(stream=None):
        x_out, y, st = tp.block_norm(x, blocks, wq, wp, gate, want_stats=True, stream=stream)
        grads = tp.block_norm_backward(dy, dxo, x_out, blocks, st, wq, wp, gate, stream=stream)
        h, cd, sc = tp.stash_pack([y], stream=stream)
        du, _ = tp.stash_backward(cd, sc, [dy], stream=stream)
        dw = tp.stash_weight_grad(cd, sc, du, stream=stream)
        return [x_out, y, st, *grads, h[0], du[0], dw[0],
                tp.qweight_matmul([y] * p, codes, scales, zeros, group=64, stream=stream)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):      # its handle exists: creating one allocates
        held = step()
    for i in range(3):
        x.copy_(norm_case(M, H, p, BF, F32, "channel", F32, False, seed=10 + i)["x"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step(), held))
