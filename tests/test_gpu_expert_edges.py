"""Routing, gradients and products at the edges of their ranges, on the GPU against float64."""
import pytest
import torch

import scaled_oracle as O
from tensor_gemm_reduction_amd import tpfuse as tp
from test_gpu_experts import BF, F8, F32, U8, cuda, gen, integer_packed, rand_u, route_of, weights

pytestmark = pytest.mark.gpu
D = torch.float64


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("E,groups,tops,k", [(32, 2, 1, 4), (32, 8, 3, 4), (256, 2, 1, 8), (256, 8, 4, 8), (1024, 2, 1, 8), (1024, 16, 5, 8)])
@pytest.mark.parametrize("size", [32.0, 1000.0, 1e4])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_of_biases_that_cancel(E, groups, tops, k, size, score):
    """A group's two largest near +B and -B, their sum near 1: the sum's error is that of its terms."""
    T, n = 16384 if E < 1024 else 4096, E // groups
    g = gen("cancel", E, size)
    # every fourth token from nearly equal sums to sums that a step of fp32 near B tells apart; the others far apart, so
    # that they do not send the wave's four to the sums in 64 bits
    x = torch.randn(T, E, generator=g)
    x[::4] = x[::4, :1] + x[::4] * torch.exp2(-20.0 * torch.rand(T // 4, 1, generator=g))
    bias = torch.full((E,), -4.0 * size)
    bias[::n], bias[1::n] = size, -size
    r = tp.expert_route(x.cuda(), k, score=score, bias=bias.cuda(), groups=groups, top_groups=tops)
    biased = O.scores(x, score) + bias.to(D)
    each = biased.view(T, groups, n)
    total = each.topk(2, dim=2).values.sum(2)
    ranked = torch.sort(total, dim=1, descending=True, stable=True)
    best = ranked.indices[:, :tops]
    allowed = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, best, True)
    value = torch.where(allowed[:, :, None], each, float("-inf")).view(T, E)
    ids = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :k]
    # Scores whose last bits differ (exp, the softmax's sum) move s + B by a step of B, up to 2^-52 B, at most: a sum of
    # two by two steps, two sums by four.  Sums that lie closer are decided by those last bits.
    decided = ranked.values[:, tops - 1] - ranked.values[:, tops] > 4 * 2.0 ** -52 * size
    assert decided.float().mean() > 0.5
    assert torch.equal(r.ids.cpu()[decided], ids.to(torch.int32)[decided])


@pytest.mark.parametrize("E,k,groups,tops,at", [
    (32, 4, 8, 2, range(1, 32, 4)), (256, 8, 8, 4, range(3, 256, 32)), (1024, 8, 16, 3, range(0, 1024, 64)),
    (64, 16, 1, 1, range(8, 12)), (64, 16, 1, 1, range(0, 4)), (61, 16, 1, 1, range(56, 61)), (256, 16, 1, 1, range(16)),
    (1024, 16, 1, 1, range(4, 1000)), (16, 12, 1, 1, range(5)), (64, 3, 1, 1, range(64)), (32, 6, 4, 2, range(8, 16))])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_with_biases_of_no_number(E, k, groups, tops, at, score):
    """NaN counts as the least: in a group's sum, beside others, and where fewer than k others remain."""
    g = gen("nan bias", E, k)
    x = torch.randn(90, E, generator=g)
    bias = torch.randn(E, generator=g) * 0.1
    bias[list(at)] = float("nan")
    r = tp.expert_route(x.cuda(), k, score=score, bias=bias.cuda(), groups=groups, top_groups=tops)
    ids = O.choose(x, k, score, bias, groups, tops, None)
    assert torch.equal(r.ids.cpu(), ids)
    for got, want in zip((r.offsets, r.src, r.pos), O.order(ids, E)):
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("E,k,groups,tops", [(64, 8, 1, 1), (61, 5, 1, 1), (32, 6, 8, 3), (256, 8, 8, 2), (1024, 16, 16, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [float("inf"), 3e38])
def test_route_with_biases_beyond_any_score(E, k, groups, tops, score, size):
    """Experts that are always or never taken, a group's sum among them that fp32 cannot hold."""
    g = gen("infinite bias", E, k)
    x = torch.randn(60, E, generator=g)
    sign = torch.randint(-1, 2, (E,), generator=g)
    bias = torch.where(sign == 0, 0.1 * torch.randn(E, generator=g), sign * size)
    for b in (bias, bias.clamp(max=1.0), bias.clamp(min=-1.0), torch.full((E,), -size)):
        r = tp.expert_route(x.cuda(), k, score=score, bias=b.cuda(), groups=groups, top_groups=tops)
        assert torch.equal(r.ids.cpu(), O.choose(x, k, score, b, groups, tops, None))


@pytest.mark.parametrize("E,k,groups,tops", [(8, 3, 1, 1), (8, 8, 1, 1), (16, 8, 1, 1), (31, 16, 1, 1), (32, 16, 1, 1),
                                             (60, 16, 1, 1), (16, 5, 4, 2), (256, 16, 8, 1), (64, 10, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_to_more_experts_than_lanes_hold(E, k, groups, tops, score, biased):
    """More experts a token than there are fours of them to choose from."""
    g = gen("few fours", E, k)
    x = torch.randn(70, E, generator=g)
    x[1] = 0.0
    x[2, k - 1:] = float("-inf")              # fewer than k that are not masked
    x[3, k:] = float("-inf")
    x[4, k - 1:] = torch.finfo(F32).min
    x[5] = torch.finfo(F32).min
    x[6] = torch.arange(E) // 2 % 5
    x[7, 0] = torch.finfo(F32).max
    bias = torch.randn(E, generator=g) * 0.1 if biased else None
    r = tp.expert_route(x.cuda(), k, score=score, bias=None if bias is None else bias.cuda(), groups=groups,
                        top_groups=tops)
    ids = O.choose(x, k, score, bias, groups, tops, None)
    assert torch.equal(r.ids.cpu(), ids)
    w = O.route_weights(x, ids, score, True, 1.0)
    assert ((r.weights.cpu().to(D) - w).abs() <= w.abs() * (O.STEP + 2.0 ** -40) + 2.0 ** -149).all()


@pytest.mark.parametrize("E", [8, 64, 130, 1024])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [True, False])
def test_softmax_of_no_number(E, biased, renorm):
    """A softmax over NaN or +inf is NaN throughout: so are the weights, of those tokens alone."""
    x = torch.randn(20, E, generator=gen("nan logit", E))
    x[3, 5] = float("nan")
    x[7, 2] = float("inf")
    bias = torch.linspace(-0.1, 0.1, E) if biased else None
    r = tp.expert_route(x.cuda(), 2, renorm=renorm, bias=None if bias is None else bias.cuda())
    bad = torch.zeros(20, 2, dtype=torch.bool)
    bad[[3, 7]] = True
    assert torch.equal(r.weights.cpu().isnan(), bad)


# ---------------------------------------------------------------------------
# the router's gradient
# ---------------------------------------------------------------------------

def confident(T, E, k, dtype):
    """Logits with one expert 8 to 14 above the others."""
    g = gen("confident", T, E, k)
    x = 0.5 * torch.randn(T, E, generator=g)
    x[torch.arange(T), torch.randint(E, (T,), generator=g)] = torch.linspace(8.0, 14.0, T) + 1.0
    return x.to(dtype), torch.randn(T, k, generator=g)


@pytest.mark.parametrize("T,E,k", [(60, 2, 1), (60, 2, 2), (70, 8, 1), (70, 64, 2), (65, 100, 3), (40, 1024, 1), (40, 1024, 16)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_a_confident_softmax(T, E, k, dtype):
    """Without renormalisation: s (1 - s) keeps its bits where s is close to 1."""
    x, dw = confident(T, E, k, dtype)
    mask = torch.arange(T) % 7 != 3
    r = tp.expert_route(x.cuda(), k, renorm=False, scale=1.7, mask=mask.cuda())
    d = tp.expert_route_backward(dw.cuda(), x.cuda(), r, renorm=False, scale=1.7).cpu().to(D)
    leaf = x.to(D).requires_grad_()
    at = r.ids.cpu().clamp(min=0).long()
    (torch.gather(torch.softmax(leaf, 1), 1, at) * 1.7 * dw.to(D) * mask[:, None]).sum().backward()
    # The terms' size without what cancels: at a chosen one 1 - s of its own and the others' s.
    s = torch.softmax(x.to(D), 1)
    one = torch.zeros(T, E, dtype=D).scatter_(1, at, 1.7 * dw.abs().to(D))
    total = (s * one).sum(1, keepdim=True)
    size = s * (one * (1.0 - s) + (total - s * one)) + s * total * (one == 0)
    # everything in 64 bits (the reference's 1 - s loses 2^-52 of 1), one rounding to fp32 and one to the result's type
    tol = leaf.grad.abs() * (O.half_step(dtype) + O.STEP) + size * 2.0 ** -40 + s * one * 2.0 ** -50
    assert ((d - leaf.grad).abs() <= tol + 2.0 ** -149).all()
    assert (d[~mask] == 0).all()


def test_gradient_of_a_softmax_of_no_number():
    x = torch.randn(8, 64, generator=gen("no number")).cuda()
    x[1, 7] = x[2] = float("nan")
    x[3, 9] = float("inf")
    x[4] = x[5, 1:] = float("-inf")
    r = tp.expert_route(x, 2, renorm=False)
    d = tp.expert_route_backward(torch.ones(8, 2).cuda(), x, r, renorm=False).cpu()
    assert torch.equal(d.isnan().all(1), torch.tensor([0, 1, 1, 1, 0, 0, 0, 0], dtype=torch.bool))
    assert (d[4:6] == 0).all() and d[[0, 6, 7]].isfinite().all()


@pytest.mark.parametrize("T,E,k", [(60, 2, 2), (70, 64, 2), (65, 100, 3), (40, 1024, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_confident_weights(T, E, k, score, dtype):
    """Renormalised weights, one close to 1: w_j (1 - w_j) keeps its bits."""
    x, dw = confident(T, E, k, dtype)
    if score == "sigmoid":
        x = (x.float() - 13.0).to(dtype)
    r = tp.expert_route(x.cuda(), k, score=score, scale=1.7)
    d = tp.expert_route_backward(dw.cuda(), x.cuda(), r, score=score, scale=1.7).cpu().to(D)
    leaf = x.to(D).requires_grad_()
    at = r.ids.cpu().long()
    w = torch.gather(O.scores(leaf, score), 1, at)
    w = 1.7 * w / w.sum(1, keepdim=True)
    (w * dw.to(D)).sum().backward()
    # w_j sum_i w_i (g_j - g_i) / scale: each weight was rounded to fp32; sums in 64 bits; a rounding to fp32 and one
    # to the result's type
    v = w.detach()
    apart = (dw.to(D)[:, :, None] - dw.to(D)[:, None, :]).abs()
    size = torch.zeros(T, E, dtype=D).scatter_(1, at, v * (v[:, None, :] * apart).sum(2) / 1.7)
    tol = leaf.grad.abs() * (O.half_step(dtype) + O.STEP) + size * 2.01 * O.STEP + 2.0 ** -50
    assert ((d - leaf.grad).abs() <= tol).all()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def extreme(g, M, K, N, kind, E=0):
    """Integer operands, scales at both ends that multiply out: (x, xs, w, ws, which results are in range)."""
    (x,), (xs,) = integer_packed(g, M, K, 1)
    (w,), (ws,) = weights(g, 1, ((E,) if E else ()) + (N, K), "f32" if kind == "f32" else "u8", integer=True)
    row = torch.tensor([252, 2, 127, 100])[torch.arange(M) % 4]
    xs[:] = row[:, None].to(U8)
    block = torch.tensor([2, 252, 127, 154])[torch.arange(O.blocks(N)) % 4]
    if kind == "u8":
        ws[:] = block[:, None].to(U8)
    else:           # 1 to 3 times the power of two, one in five of them negative
        sign = torch.where(torch.rand(ws.shape, generator=g) < 0.2, -1.0, 1.0)
        ws.copy_(ws * sign * torch.exp2(block.float() - 127.0)[:, None])
    column = torch.repeat_interleave(block, 128)[:N]
    return x, xs, w, ws, (row[:, None] + column[None, :] - 254).abs() <= 14


# few rows; tiles of 128 x 128; of 256 x 256 (powers of two, bf16)
@pytest.mark.parametrize("M,K,N", [(9, 272, 520), (40, 144, 520), (700, 272, 1032), (3600, 144, 3592)])
@pytest.mark.parametrize("kind", ["u8", "f32"])
@pytest.mark.parametrize("out", [BF, F32])
def test_extreme_scales_of_products(M, K, N, kind, out):
    x, xs, w, ws, ok = extreme(gen("ends", M), M, K, N, kind)
    y = tp.fp8_matmul([x.cuda()], [xs.cuda()], [w.cuda()], [ws.cuda()], out_dtype=out).cpu()
    want = (O.values(x, xs) @ O.weight(w, ws).t()).to(out)
    assert torch.equal(y[ok], want[ok])


@pytest.mark.parametrize("T,E,k,K,N", [(40, 5, 2, 144, 520), (4000, 3, 2, 144, 1032), (3000, 60, 4, 144, 1032)])
@pytest.mark.parametrize("kind", ["u8", "f32"])
@pytest.mark.parametrize("out", [BF, F32])
def test_extreme_scales_of_experts(T, E, k, K, N, kind, out):
    g = gen("ends", T, E)
    r = route_of(g, T, E, k)
    x, xs, w, ws, ok = extreme(g, T * k, K, N, kind, E)
    y = tp.expert_matmul([x.cuda()], [xs.cuda()], [w.cuda()], [ws.cuda()], tp.ExpertRoute(*(t.cuda() for t in r)),
                         out_dtype=out).cpu()
    xv = O.values(x, xs)
    for e in range(E):
        at = slice(int(r.offsets[e]), int(r.offsets[e + 1]))
        want = (xv[at] @ O.weight(w[e], ws[e]).t()).to(out)
        assert torch.equal(y[at][ok[at]], want[ok[at]])


@pytest.mark.parametrize("R,C", [(264, 392), (3600, 3592)])
@pytest.mark.parametrize("out", [BF, F32])
def test_extreme_scales_of_weight_gradients(R, C, out):
    g = gen("ends", R)
    (a,), (as_,) = integer_packed(g, R, 256, 1)
    (b,), (bs,) = integer_packed(g, C, 256, 1)
    row, col = torch.tensor([252, 2, 127, 100])[torch.arange(R) % 4], torch.tensor([2, 252, 127])[torch.arange(C) % 3]
    as_[:], bs[:] = row[:, None].to(U8), col[:, None].to(U8)
    ok = (row[:, None] + col[None, :] - 254).abs() <= 14
    dw = tp.fp8_weight_grad([a.cuda()], [as_.cuda()], [b.cuda()], [bs.cuda()], out_dtype=out)[0].cpu()
    want = (O.values(a, as_) @ O.values(b, bs).t()).to(out)
    assert torch.equal(dw[ok], want[ok])


@pytest.mark.parametrize("M,K,N", [(9, 128, 520), (700, 128, 1032)])
@pytest.mark.parametrize("out", [BF, F32])
def test_factors_that_are_special(M, K, N, out):
    """fp32 scales of zero, below the least normal number, infinite and NaN, each in its own columns."""
    g = gen("special", M)
    (x,), (xs,), (w,), (ws,) = *integer_packed(g, M, K, 1), *weights(g, 1, (N, K), "f32", integer=True)
    sign = torch.where(torch.arange(M)[:, None] % 2 == 0, 1.0, -1.0)
    x, w = (sign * x.float().abs().clamp(min=1.0)).to(F8), w.float().abs().clamp(min=1.0).to(F8)    # no sum is 0
    xs[:] = 127
    xs[1] = 250
    factors = (1.0, 0.0, 3 * 2.0 ** -140, float("inf"), float("nan"))
    ws[:5, 0] = torch.tensor(factors)
    y = tp.fp8_matmul([x.cuda()], [xs.cuda()], [w.cuda()], [ws.cuda()], out_dtype=out).cpu()
    part = O.values(x, xs) @ w.to(D).t()
    for i, f in enumerate(factors):
        at = slice(128 * i, min(128 * (i + 1), N))
        want = (part[:, at] * f).to(out)
        rows = [1] if f == 3 * 2.0 ** -140 else [m for m in range(M) if m != 1 or i == 1]   # results below fp32's range
        assert torch.equal(y[rows][:, at].nan_to_num(nan=1e30, posinf=2e30, neginf=-2e30),
                           want[rows].nan_to_num(nan=1e30, posinf=2e30, neginf=-2e30))


# workgroups up to the compute units' number and above it, of as many blocks as waves and fewer
@pytest.mark.parametrize("p,M,K,N", [(1, 3, 1040, 8192), (1, 16, 1040, 8200), (2, 1, 528, 8264), (2, 16, 400, 8264), (1, 5, 400, 520),
                                     (1, 33, 1040, 264), (1, 30, 1040, 8200), (3, 64, 400, 2056)])
@pytest.mark.parametrize("kind", ["u8", "f32"])
@pytest.mark.parametrize("out", [BF, F32])
def test_few_rows_of_wide_results(p, M, K, N, kind, out):
    g = gen("wide", p, M, K)
    x, xs = integer_packed(g, M, K, p)
    w, ws = weights(g, p, (N, K), kind, integer=True)
    y = tp.fp8_matmul(cuda(x), cuda(xs), cuda(w), cuda(ws), out_dtype=out)
    want = sum(O.values(x[k], xs[k]) @ O.weight(w[k], ws[k]).t() for k in range(p))
    assert torch.equal(y.cpu(), want.to(out))


def gelu_operands(rows, N):
    """Operands whose sums are exact, i + j / 16 + n / 256 from -13 to 4: (x, xs, w, ws, the sums)."""
    x, w = torch.zeros(rows, 16), torch.zeros(N, 16)
    whole, part = torch.arange(rows) % 17 - 13, torch.arange(rows) // 17 % 16
    x[:, 0], x[:, 1], x[:, 2] = whole, part, 1.0
    w[:, 0], w[:, 1], w[:, 2] = 1.0, 1.0 / 16, torch.arange(N) % 16 / 256
    one = lambda *s: torch.full(s, 127, dtype=U8)
    u = x.to(D) @ w.to(D).t()
    assert torch.equal(x.to(F8).to(D) @ w.to(F8).to(D).t(), u)
    return x.to(F8), one(rows, 4), w.to(F8), one(O.blocks(N), 1), u


@pytest.mark.parametrize("M,N", [(272, 16), (816, 1032)])
@pytest.mark.parametrize("out", [BF, F32])
def test_gelu_of_far_values(M, N, out):
    """Relative to GeLU itself, of few rows and on tiles.  fp32: 16 half steps of fp32 (2^-20), for the reciprocal, exp2
    and products and sums of their fp32 values; bf16: 2^-16 for the square's rounding in the exponent."""
    x, xs, w, ws, u = gelu_operands(M, N)
    y = tp.fp8_matmul([x.cuda()], [xs.cuda()], [w.cuda()], [ws.cuda()], gelu=True, out_dtype=out).cpu().to(D)
    want = O.gelu(u)
    own = 2.0 ** -20 if out == F32 else O.half_step(BF) + 2.0 ** -16
    assert ((y - want).abs() <= want.abs() * own).all()


def test_gelu_of_extreme_values():
    x = torch.zeros(9, 16)
    x[:, 0] = torch.tensor([448.0, -448.0, 0.0, -0.0, 20.0, -20.0, 8.0, -8.0, 1.0])
    x, w = x.to(F8), torch.eye(8, 16).to(F8)
    for out in (BF, F32):
        for scale in (127, 245):            # 2^118 of them: beyond what the square can hold
            xs, ws = torch.full((9, 4), scale, dtype=U8), torch.full((1, 1), 127, dtype=U8)
            y = tp.fp8_matmul([x.cuda()], [xs.cuda()], [w.cuda()], [ws.cuda()], gelu=True, out_dtype=out).cpu().to(D)[:, 0]
            want = O.gelu(torch.ldexp(x[:, 0].to(D), torch.tensor(scale - 127)))
            assert ((y - want).abs() <= want.abs() * (2.0 ** -16 + O.half_step(out)) + 1e-37).all()


# ---------------------------------------------------------------------------
# sums in fp32
# ---------------------------------------------------------------------------

def cancelling(rows, K, first=True):
    """Rows whose products with the other operand's are 448 * 448, -448 * 448 and 6, side by side, and zeros."""
    codes = torch.zeros(rows, K)
    if first:
        for m in range(rows):
            codes[m, 3 * (m % (K // 3)):][:3] = torch.tensor([448.0, 448.0, 6.0])
    else:
        codes[:] = torch.tensor([448.0, -448.0, 1.0])[torch.arange(K) % 3]
    return codes.to(F8), torch.full((rows, O.width(K)), 127, dtype=U8)


@pytest.mark.parametrize("M,N", [(9, 264), (40, 264), (700, 1032), (3600, 3592)])
@pytest.mark.parametrize("kind", ["u8", "f32"])
def test_cancelling_products(M, N, kind):
    (x, xs), (w, _) = cancelling(M, 256), cancelling(N, 256, False)
    ws = torch.full((O.blocks(N), 2), 127, dtype=U8) if kind == "u8" else torch.ones(O.blocks(N), 2)
    args = [[t.cuda()] for t in (x, xs, w, ws)]
    assert (tp.fp8_matmul(*args, fp32_sums=True) == 6).all()
    assert (tp.fp8_matmul(*args, out_dtype=F32) == 6).all()
    # 13 places below the largest of eight products
    assert ((tp.fp8_matmul(*args).double() - 6).abs() <= 2.0 ** -10 * (2 * 448 * 448 + 6) + 8 * O.half_step(BF)).all()
    if M <= 40:
        assert (tp.fp8_matmul(*args) == 6).all()


@pytest.mark.parametrize("T,E,k,N", [(10, 8, 2, 264), (40, 5, 2, 264), (3000, 60, 4, 1032)])
@pytest.mark.parametrize("kind", ["u8", "f32"])
def test_cancelling_products_of_experts(T, E, k, N, kind):
    r = tp.ExpertRoute(*(t.cuda() for t in route_of(gen("cancel", T), T, E, k)))
    (x, xs), (w, _) = cancelling(T * k, 256), cancelling(N, 256, False)
    ws = torch.full((E, O.blocks(N), 2), 127, dtype=U8) if kind == "u8" else torch.ones(E, O.blocks(N), 2)
    w = w.expand(E, -1, -1).contiguous()
    for fine in [True] if T > 10 else [True, False]:           # of few rows always
        y = tp.expert_matmul([x.cuda()], [xs.cuda()], [w.cuda()], [ws.cuda()], r, fp32_sums=fine)
        assert y.dtype == BF and (y == 6).all()


@pytest.mark.parametrize("R,C", [(130, 24), (2000, 2056)])
def test_cancelling_weight_gradients(R, C):
    (a, as_), (b, bs) = cancelling(R, 256), cancelling(C, 256, False)
    dw, = tp.fp8_weight_grad([a.cuda()], [as_.cuda()], [b.cuda()], [bs.cuda()], out_dtype=BF, fp32_sums=True)
    assert dw.dtype == BF and (dw == 6).all()
    # two experts of 128 rows each
    r = tp.ExpertRoute(*(t.cuda() for t in (torch.arange(256).int()[:, None] // 128, torch.ones(256, 1),
                                            torch.tensor([0, 128, 256]).int(), torch.arange(256).int(),
                                            torch.arange(256).int()[:, None])))
    Mt = tp.fp8_columns(256, 2)
    (a, as_), (b, bs) = cancelling(R, Mt), cancelling(C, Mt, False)
    a[:, 126:] = 0
    a[:, 128:131] = torch.tensor([448.0, 448.0, 6.0]).roll(-128 % 3).to(F8)
    dw, = tp.expert_weight_grad([a.cuda()], [as_.cuda()], [b.cuda()], [bs.cuda()], r, out_dtype=BF, fp32_sums=True)
    av, bv = a.to(D), b.to(D)
    assert torch.equal(dw.cpu(), torch.stack([av[:, :128] @ bv[:, :128].t(), av[:, 128:256] @ bv[:, 128:256].t()]).to(BF))


@pytest.mark.parametrize("p,M,K,N", [(2, 16, 272, 136), (1, 64, 528, 96), (2, 700, 400, 1032), (1, 3600, 144, 3592)])
@pytest.mark.parametrize("kind", ["u8", "f32"])
@pytest.mark.parametrize("act", [False, True])
def test_sums_in_fp32(p, M, K, N, kind, act):
    """bf16 results without the 8-bit instructions' 2^-10: of few rows always, of others on request."""
    g = gen("fine", p, M, K)
    x, xs = zip(*(O.pack(u) for u in rand_u(g, M, K, p)))
    x, xs = [t.to(F8) for t in x], [t.to(U8) for t in xs]
    w, ws = weights(g, p, (N, K), kind)
    ws = [t - 16 if kind == "u8" else t / 4096 for t in ws]
    y = tp.fp8_matmul(cuda(x), cuda(xs), cuda(w), cuda(ws), gelu=act, fp32_sums=M > 64).cpu().to(D)
    xv, wv = [O.values(*t) for t in zip(x, xs)], [O.weight(*t) for t in zip(w, ws)]
    want, size = sum(a @ b.t() for a, b in zip(xv, wv)), sum(a.abs() @ b.abs().t() for a, b in zip(xv, wv))
    # p K roundings to fp32 of sums up to `size`, GeLU's slope (below 1.13) and its own roundings, one rounding to bf16
    slack = size * p * K * 2.0 ** -23
    if act:
        slack, want = 1.13 * slack + want.abs() * 2.0 ** -20, O.gelu(want)
    assert ((y - want).abs() <= want.abs() * O.half_step(BF) + slack * (1 + O.half_step(BF))).all()
