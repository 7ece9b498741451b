"""8-bit products and routing where other kernels, the largest sizes and 64-bit offsets come in.
Integer operands: compared exactly.  Tolerances of the others as in test_gpu_experts."""
import pytest
import torch

import scaled_oracle as O
from tensor_gemm_reduction_amd import tpfuse as tp
from test_gpu_experts import BF, F8, F32, U8, check_sum, cuda, gen, integer_packed, rand_u, route_of, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p,M,K,N", [(2, 700, 400, 1032), (3, 1001, 144, 520), (1, 1100, 1168, 520), (1, 513, 16, 1096)])
@pytest.mark.parametrize("kind", ["u8", "f32"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("act", [False, True])
def test_matmul_of_many_rows(p, M, K, N, kind, out, act):
    g = gen("mid", p, M, K, N)
    x, xs = zip(*(O.pack(u) for u in rand_u(g, M, K, p)))
    x, xs = [t.to(F8) for t in x], [t.to(U8) for t in xs]
    w, ws = weights(g, p, (N, K), kind)
    ws = [t - 16 if kind == "u8" else t / 4096 for t in ws]
    y = tp.fp8_matmul(cuda(x), cuda(xs), cuda(w), cuda(ws), gelu=act, out_dtype=out)
    xv, wv = [O.values(*t) for t in zip(x, xs)], [O.weight(*t) for t in zip(w, ws)]
    check_sum(y, sum(a @ b.t() for a, b in zip(xv, wv)), sum(a.abs() @ b.abs().t() for a, b in zip(xv, wv)), p * K, out, act)


def test_matmul_of_many_rows_with_gelu_on_large_tiles():
    g = gen("biggelu")
    M, K, N = 3600, 144, 3600
    (x, xs), (w, ws) = integer_packed(g, M, K, 1), weights(g, 1, (N, K), "u8", integer=True)
    ws = [t - 7 for t in ws]
    y = tp.fp8_matmul(cuda(x), cuda(xs), cuda(w), cuda(ws), gelu=True)
    xv, wv = O.values(x[0], xs[0]), O.weight(w[0], ws[0])
    check_sum(y, xv @ wv.t(), xv.abs() @ wv.abs().t(), K, BF, True)


# (T, E, k, K, N): tiles of 128 x 128, 256 x 256 and 128 x 256, rows of no expert
@pytest.mark.parametrize("T,E,k,K,N", [(4000, 3, 2, 144, 1032), (8000, 3, 2, 272, 1016), (3000, 60, 4, 144, 1032), (4000, 60, 4, 144, 2056)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("act", [False, True])
def test_expert_matmul_of_many_rows(T, E, k, K, N, gather, act):
    g = gen("bigexperts", T, E, k, K)
    r = route_of(g, T, E, k, 0.5, True)
    x, xs = integer_packed(g, T if gather else T * k, K, 1)
    w, ws = weights(g, 1, (E, N, K), "u8", integer=True)
    ws = [t - 7 for t in ws] if act else ws
    Y = torch.full((T * k, N), float("nan"), dtype=BF).cuda()
    y = tp.expert_matmul(cuda(x), cuda(xs), cuda(w), cuda(ws), tp.ExpertRoute(*(t.cuda() for t in r)), gather=gather, gelu=act, Y=Y)
    want, size = (torch.zeros(T * k, N, dtype=torch.float64) for _ in range(2))
    xv = O.values(x[0], xs[0])
    for e in range(E):
        lo, hi = int(r.offsets[e]), int(r.offsets[e + 1])
        rows, wv = xv[r.src[lo:hi].long() // k if gather else slice(lo, hi)], O.weight(w[0][e], ws[0][e])
        want[lo:hi], size[lo:hi] = rows @ wv.t(), rows.abs() @ wv.abs().t()
    if act:
        check_sum(y, want, size, K, BF, True)
    else:
        assert torch.equal(y.cpu(), want.to(BF))
    assert (y[int(r.offsets[-1]):] == 0).all()


@pytest.mark.parametrize("T,E,k,R,C,p", [(1500, 16, 2, 1000, 1032, 1), (900, 5, 2, 776, 520, 4), (2500, 2, 1, 2048, 2048, 2)])
def test_expert_weight_grad_of_large_tiles(T, E, k, R, C, p):
    g = gen("bigdw", T, E)
    r = route_of(g, T, E, k, 1.0, True)
    Mt = O.columns(T * k, E)
    (a, as_), (b, bs) = integer_packed(g, R, Mt, p), integer_packed(g, C, Mt, p)
    dW = [torch.full((E, R, C), float("nan"), dtype=BF).cuda() for _ in range(p)]
    tp.expert_weight_grad(cuda(a), cuda(as_), cuda(b), cuda(bs), tp.ExpertRoute(*(t.cuda() for t in r)), dW=dW)
    for j in range(p):
        av, bv, col = O.values(a[j], as_[j]), O.values(b[j], bs[j]), 0
        for e in range(E):
            n = O.blocks(int(r.offsets[e + 1] - r.offsets[e])) * 128
            assert torch.equal(dW[j][e].cpu(), (av[:, col:col + n] @ bv[:, col:col + n].t()).to(BF))
            col += n


@pytest.mark.parametrize("M,N", [(9, 264), (40, 264), (700, 1032), (3600, 3592)])
@pytest.mark.parametrize("out", [BF, F32])
def test_scale_of_no_number(M, N, out):
    """255 in a row's or a weight's scales is NaN, in every kernel, and reaches its own results alone."""
    g = gen("nan scale", M)
    K = 272
    (x, xs), (w, ws) = integer_packed(g, M, K, 1), weights(g, 1, (N, K), "u8", integer=True)
    want = (O.values(x[0], xs[0]) @ O.weight(w[0], ws[0]).t()).to(out)
    xs[0][5, 1] = 255
    ws[0][1, 2] = 255
    y = tp.fp8_matmul(cuda(x), cuda(xs), cuda(w), cuda(ws), out_dtype=out).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[5], bad[:, 128:256] = True, True
    assert torch.equal(y.isnan(), bad)
    assert torch.equal(y[~bad], want[~bad])


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("E,k,groups,tops", [(1024, 16, 1, 1), (1024, 16, 16, 2), (1000, 8, 8, 3), (250, 8, 10, 4), (48, 3, 8, 2), (62, 5, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_route_of_equal_logits(E, k, groups, tops, score, dtype):
    """All equal, few different values, and one expert above: more equals than a list holds."""
    g = gen("equal", E, k)
    x = torch.cat([torch.zeros(3, E), torch.randint(0, 3, (40, E), generator=g).float(),
                   torch.nn.functional.one_hot(torch.randint(0, E, (10,), generator=g), E).float()]).to(dtype)
    wide = torch.randint(0, 2, (E + 1,), generator=g).float()
    odd = torch.empty(E + 1).cuda()
    odd.copy_(wide)
    for bias in (None, odd[1:]):              # four bytes past 16
        r = tp.expert_route(x.cuda(), k, score=score, bias=bias, groups=groups, top_groups=tops)
        ids = O.choose(x, k, score, None if bias is None else wide[1:], groups, tops, None)
        assert torch.equal(r.ids.cpu(), ids)
        w = O.route_weights(x, ids, score, True, 1.0)
        assert ((r.weights.cpu().double() - w).abs() <= w.abs() * (O.STEP + 2.0 ** -45)).all()


@pytest.mark.parametrize("T,E,k", [(1, 5, 2), (200, 61, 8), (1100, 129, 8), (70, 250, 16), (40, 517, 9), (30, 1023, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_of_odd_numbers_of_experts(T, E, k, score, dtype, renorm):
    """Rows of logits that start at any element; values past the last expert's belong to the next row."""
    g = gen("odd", T, E)
    x = (3 * torch.randn(T, E, generator=g)).to(dtype)
    x[:, 0] += 4.0 * (torch.rand(T, generator=g) < 0.5).to(dtype)        # beside the end of the row before
    for bias in (None, torch.randn(E, generator=g) * 0.2):
        r = tp.expert_route(x.cuda(), k, score=score, renorm=renorm, bias=None if bias is None else bias.cuda())
        ids = O.choose(x, k, score, bias, 1, 1, None)
        assert torch.equal(r.ids.cpu(), ids)
        for got, want in zip((r.offsets, r.src, r.pos), O.order(ids, E)):
            assert torch.equal(got.cpu(), want)
        w = O.route_weights(x, ids, score, renorm, 1.0)
        assert ((r.weights.cpu().double() - w).abs() <= w.abs() * (O.STEP + 2.0 ** -45)).all()


def test_two_graphs_share_a_workspace():
    T, E, k = 5000, 64, 4
    side = torch.cuda.Stream()
    ws = torch.empty(tp.load().tpf_expert_route_ws(T, E), dtype=U8, device="cuda")
    xs = [torch.randn(T, E, generator=gen("graph", i)).cuda() for i in range(2)]
    side.wait_stream(torch.cuda.current_stream())
    tp.expert_route(xs[0], k, ws=ws, stream=side)
    side.synchronize()
    graphs, routes = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for x, graph in zip(xs, graphs):
        with torch.cuda.graph(graph, stream=side):
            routes.append(tp.expert_route(x, k, ws=ws))
    for i in range(3):
        for x, graph, r in zip(xs, graphs, routes):
            x.copy_(torch.randn(T, E, generator=gen("again", i)))
            graph.replay()
        torch.cuda.synchronize()
        for x, r in zip(xs, routes):
            assert all(torch.equal(a, b) for a, b in zip(r, tp.expert_route(x, k)))


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------

def test_rows_past_two_to_the_thirty():
    """Packing and the product of 1.1e9 rows: 35 GB of activations, 8.6e6 tiles."""
    M, K, N = 1_100_000_000, 16, 8
    at = torch.tensor([0, 1, 70_000, 2 ** 27 + 3, 2 ** 28 + 130, 2 ** 30 - 1, 2 ** 30, M - 129, M - 1])
    g = gen("long")
    some = torch.randint(-6, 7, (len(at), K), generator=g).bfloat16()
    u = torch.zeros(M, K, dtype=BF, device="cuda")
    u[at.cuda()] = some.cuda()
    codes, scales, _, _ = tp.fp8_pack([u])
    del u
    w, ws = weights(g, 1, (N, K), "u8", integer=True)
    y = tp.fp8_matmul(codes, scales, cuda(w), cuda(ws))
    assert torch.equal(y[at.cuda()].cpu(), (some.double() @ O.weight(w[0], ws[0]).t()).to(BF))
    for i in range(0, M, 1 << 28):
        assert int((y[i:i + (1 << 28)] != 0).any(1).sum()) == int(((at >= i) & (at < i + (1 << 28))).sum())


def test_experts_rows_past_four_gigabytes():
    """70000 rows of 65536: products, transposes, weight gradients, sums and their gradients."""
    T, E, k, K, N = 35_000, 4, 2, 65_536, 64
    g = gen("wide")
    r = tp.expert_route(torch.randn(T, E, generator=g).cuda(), k)
    offsets = r.offsets.cpu()
    rows = torch.randint(-2, 3, (T * k, K), dtype=torch.int8, device="cuda").to(BF)
    codes, scales, turned, turned_scales = tp.fp8_pack([rows], columns=True, route=r)
    w, ws = weights(g, 1, (E, N, K), "u8", integer=True)
    y = tp.expert_matmul(codes, scales, cuda(w), cuda(ws), r, out_dtype=F32)
    del codes, scales
    for row in (0, 1, 32_767, 32_769, 65_535, 65_537, 69_999):
        e = int(torch.searchsorted(offsets, row, right=True)) - 1
        want = O.weight(w[0][e], ws[0][e]) @ rows[row].cpu().double()
        assert torch.equal(y[row].cpu().double(), want)         # integers below 2^24
    small = torch.randint(-2, 3, (T * k, N), dtype=torch.int8, device="cuda").to(BF)
    _, _, st, ss = tp.fp8_pack([small], rows=False, columns=True, route=r)
    dw, = tp.expert_weight_grad(turned, turned_scales, st, ss, r)
    del turned, turned_scales
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        for c in (0, 255, 256, 40_001, K - 1):
            assert torch.equal(dw[e, c].cpu().double(), small[lo:hi].cpu().double().t() @ rows[lo:hi, c].cpu().double())
    del dw
    y = tp.expert_combine(rows, r, out_dtype=F32)
    tokens = [0, 1, 16_384, 20_000, T - 1]
    dy = torch.zeros(T, K, dtype=BF, device="cuda")
    dy[tokens] = torch.randint(-2, 3, (len(tokens), K), dtype=torch.int8, device="cuda").to(BF)
    drows, dw = tp.expert_combine_backward(dy, rows, r)
    for t in tokens:
        own, wt = rows[r.pos[t].long()].cpu().double(), r.weights[t].cpu().double()
        want = (own * wt[:, None]).sum(0)
        # two products and a sum of fp32 terms
        assert ((y[t].cpu().double() - want).abs() <= 2 * O.STEP * (own.abs() * wt[:, None]).sum(0)).all()
        d = dy[t].cpu().double()
        assert torch.equal(dw[t].cpu().double(), own @ d)        # integers below 2^24
        grad = drows[r.pos[t].long()].cpu().double()
        # the product in fp32, then bf16
        assert ((grad - wt[:, None] * d).abs() <= (wt[:, None] * d).abs() * (O.half_step(BF) + 2 * O.STEP)).all()
    assert int((drows != 0).any(1).sum()) == k * len(tokens)
