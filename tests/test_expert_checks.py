"""Refusals of the 8-bit Linears and the MLP block of experts, and the oracle's
gradients against differences.  No GPU: the C ABI is called with a NULL handle and
pointers that are never followed, the binding with host tensors."""
import pytest
import torch

import scaled_oracle as O
from tensor_gemm_reduction_amd import tpfuse as tp

A, MIS8, MIS2, ODD = 0x1000, 0x1008, 0x1002, 0x1001
BF, U8, F8, I32, F32 = torch.bfloat16, torch.uint8, torch.float8_e4m3fn, torch.int32, torch.float32
INVALID, SHAPE, ALIGN, WS, UNSUP = (tp.ERR_INVALID_ARG, tp.ERR_SHAPE, tp.ERR_ALIGNMENT, tp.ERR_WORKSPACE,
                                    tp.ERR_UNSUPPORTED)


def arr(v, n=2):
    return None if v is None else tp.ptr_array(v if isinstance(v, list) else [v] * n)


def pack(p=2, M=4, K=64, u=A, codes=A, scales=A, ct=A, st=A, E=0, offsets=A, src=A, top=0):
    return tp.load().tpf_scaled_pack(None, p, M, K, arr(u), arr(codes), arr(scales), arr(ct), arr(st), E, offsets, src,
                                     top, None)


def mm(p=2, M=4, K=64, N=8, x=A, xs=A, w=A, ws=ODD, kind=0, y=A, yt=0):
    return tp.load().tpf_scaled_matmul(None, p, M, K, N, arr(x), arr(xs), arr(w), arr(ws), kind, 0, y, yt, None)


def grad(p=2, M=128, R=16, C=8, a=A, as_=A, b=A, bs=A, dw=A, dt=0):
    return tp.load().tpf_scaled_weight_grad(None, p, M, R, C, arr(a), arr(as_), arr(b), arr(bs), arr(dw), dt, None)


def emm(p=2, R=8, K=64, N=8, E=4, x=A, xs=A, w=A, ws=ODD, kind=0, offsets=A, src=A, top=2, y=A, yt=0):
    return tp.load().tpf_expert_matmul(None, p, R, K, N, E, arr(x), arr(xs), arr(w), arr(ws), kind, offsets, src, top, 0,
                                       y, yt, None)


def egrad(p=2, M=128, R=16, C=8, E=4, a=A, as_=A, b=A, bs=A, offsets=A, dw=A, dt=0):
    return tp.load().tpf_expert_weight_grad(None, p, M, R, C, E, arr(a), arr(as_), arr(b), arr(bs), offsets, arr(dw), dt,
                                            None)


def route(T=4, E=8, k=2, x=A, xt=0, score=0, bias=A, groups=1, tops=1, scale=1.0, ids=A, w=A, off=A, src=A, pos=A, ws=A,
          nb=1 << 20):
    return tp.load().tpf_expert_route(None, T, E, k, x, xt, score, bias, groups, tops, 1, scale, None, ids, w, off, src,
                                      pos, ws, nb, None)


def rgrad(T=4, E=8, k=2, x=A, xt=0, score=0, scale=1.0, ids=A, w=A, dw=A, d=A):
    return tp.load().tpf_expert_route_backward(None, T, E, k, x, xt, score, 1, scale, ids, w, dw, d, None)


def comb(T=4, k=2, H=8, rows=A, rt=0, w=A, pos=A, y=A, yt=0):
    return tp.load().tpf_expert_combine(None, T, k, H, rows, rt, w, pos, y, yt, None)


def cgrad(T=4, k=2, H=8, E=4, dy=A, yt=0, rows=A, rt=0, w=A, pos=A, off=A, dr=A, dw=A):
    return tp.load().tpf_expert_combine_backward(None, T, k, H, E, dy, yt, rows, rt, w, pos, off, dr, dw, None)


@pytest.mark.parametrize("call,kw,code", [
    (pack, dict(p=0), SHAPE), (pack, dict(p=17), SHAPE), (pack, dict(M=0), SHAPE), (pack, dict(K=24), ALIGN),
    (pack, dict(K=1 << 23), UNSUP), (pack, dict(u=None), INVALID), (pack, dict(u=[A, MIS8]), ALIGN),
    (pack, dict(codes=None), INVALID), (pack, dict(codes=None, scales=None, ct=None, st=None), INVALID),
    (pack, dict(st=None), INVALID), (pack, dict(codes=MIS8), ALIGN), (pack, dict(scales=MIS2), ALIGN),
    (pack, dict(ct=MIS8), ALIGN), (pack, dict(st=ODD), ALIGN), (pack, dict(E=1025), UNSUP), (pack, dict(E=-1), UNSUP),
    (pack, dict(E=4, offsets=None), INVALID), (pack, dict(E=4, top=17), SHAPE), (pack, dict(E=4, top=2, src=None), INVALID),
    (pack, dict(E=4, top=2, src=MIS2), ALIGN), (pack, dict(M=(1 << 22) + 1), UNSUP), (pack, dict(K=1 << 21), UNSUP),
    (mm, dict(p=0), SHAPE), (mm, dict(M=0), SHAPE), (mm, dict(K=8), ALIGN), (mm, dict(N=12), ALIGN), (mm, dict(N=0), SHAPE),
    (mm, dict(N=(1 << 20) + 8), UNSUP), (mm, dict(kind=2), INVALID), (mm, dict(yt=3), INVALID), (mm, dict(x=MIS8), ALIGN),
    (mm, dict(xs=MIS2), ALIGN), (mm, dict(w=[A, 0]), INVALID), (mm, dict(kind=1), ALIGN), (mm, dict(ws=None), INVALID),
    (mm, dict(y=None), INVALID), (mm, dict(y=MIS8), ALIGN), (mm, dict(M=(1 << 31) - 1, N=1 << 20), UNSUP),
    (grad, dict(M=130), ALIGN), (grad, dict(M=144), SHAPE), (grad, dict(R=0), SHAPE), (grad, dict(C=4), ALIGN),
    (grad, dict(a=MIS8), ALIGN), (grad, dict(as_=MIS2), ALIGN), (grad, dict(bs=[A, 0]), INVALID), (grad, dict(dw=MIS8), ALIGN),
    (grad, dict(dt=7), INVALID),
    (emm, dict(E=0), UNSUP), (emm, dict(E=1025), UNSUP), (emm, dict(offsets=None), INVALID), (emm, dict(top=3), SHAPE),
    (emm, dict(top=-1), SHAPE), (emm, dict(src=None), INVALID), (emm, dict(R=0), SHAPE), (emm, dict(offsets=MIS2), ALIGN),
    (emm, dict(R=1 << 26, K=64, top=1), UNSUP), (emm, dict(y=MIS8), ALIGN),
    (egrad, dict(E=0), UNSUP), (egrad, dict(offsets=None), INVALID), (egrad, dict(M=64), SHAPE), (egrad, dict(dw=[A, 0]), INVALID),
    (route, dict(T=0), SHAPE), (route, dict(E=1025), UNSUP), (route, dict(k=0), SHAPE), (route, dict(k=9), SHAPE),
    (route, dict(k=17, E=64), SHAPE), (route, dict(xt=2), INVALID), (route, dict(score=2), INVALID),
    (route, dict(scale=0.0), INVALID), (route, dict(scale=float("nan")), INVALID), (route, dict(scale=float("inf")), INVALID),
    (route, dict(groups=0), SHAPE), (route, dict(groups=3), SHAPE), (route, dict(groups=17, E=34), SHAPE),
    (route, dict(groups=2, tops=3), SHAPE), (route, dict(groups=2, tops=0), SHAPE), (route, dict(groups=4, tops=1, k=3), SHAPE),
    (route, dict(x=MIS8), ALIGN), (route, dict(bias=MIS2), ALIGN), (route, dict(ids=None), INVALID), (route, dict(w=None), INVALID),
    (route, dict(off=MIS2), ALIGN), (route, dict(src=None), INVALID), (route, dict(pos=None), INVALID), (route, dict(ws=None), WS),
    (route, dict(nb=16), WS), (route, dict(T=1 << 30, k=8), SHAPE),
    (rgrad, dict(k=0), SHAPE), (rgrad, dict(scale=0.0), INVALID), (rgrad, dict(dw=None), INVALID), (rgrad, dict(d=MIS8), ALIGN),
    (comb, dict(H=12), ALIGN), (comb, dict(k=17), SHAPE), (comb, dict(rt=5), INVALID), (comb, dict(rows=MIS8), ALIGN),
    (comb, dict(w=None), INVALID), (comb, dict(pos=MIS2), ALIGN), (comb, dict(y=None), INVALID), (comb, dict(T=1 << 30, k=2), SHAPE),
    (cgrad, dict(E=0), UNSUP), (cgrad, dict(dy=MIS8), ALIGN), (cgrad, dict(off=None), INVALID), (cgrad, dict(dr=MIS8), ALIGN),
    (cgrad, dict(dw=None), INVALID), (cgrad, dict(H=0), SHAPE),
])
def test_refusals(call, kw, code):
    assert call(**kw) == code
    assert tp.load().tpf_last_error()


@pytest.mark.parametrize("call", [pack, mm, grad, emm, egrad, route, rgrad, comb, cgrad])
def test_good_arguments_end_at_the_handle(call):
    assert call() == INVALID
    assert "handle" in tp.load().tpf_last_error().decode()


def test_sizes():
    assert [tp.fp8_scale_width(n) for n in (16, 128, 512, 528, 1024)] == [4, 4, 4, 8, 8]
    assert [tp.fp8_columns(n) for n in (1, 128, 129)] == [128, 128, 256]
    for R, E in ((1, 1), (1, 64), (7, 4), (1000, 8), (4096, 60), (5, 1024)):
        assert tp.fp8_columns(R, E) == O.columns(R, E)
        # no loads need more: the worst has as many experts with one row as there can be
        few = min(E, R)
        assert tp.fp8_columns(R, E) >= 128 * (few - 1) + O.columns(R - few + 1)
    assert tp.fp8_columns(10, 1025) == 0
    lib = tp.load()
    assert lib.tpf_expert_route_ws(1, 8) > 0 and lib.tpf_expert_route_ws(0, 8) == 0 and lib.tpf_expert_route_ws(4, 2000) == 0
    assert lib.tpf_expert_route_ws(16384, 256) == 256 * 256 * 2


def host(*shape, dtype=BF):
    return torch.zeros(shape).to(dtype)


ROUTE = tp.ExpertRoute(host(4, 2, dtype=I32), host(4, 2, dtype=F32), host(9, dtype=I32), host(8, dtype=I32),
                       host(4, 2, dtype=I32))
X, XS, W, WSC = host(4, 64, dtype=F8), host(4, 4, dtype=U8), host(8, 64, dtype=F8), host(1, 1, dtype=U8)


@pytest.mark.parametrize("bad,what", [(host(64), "has 1 dimensions"), (None, "is not a tensor"), (host(2, 4, 64), "has 3 dim")])
@pytest.mark.parametrize("name,call", [
    (r"u\[0\]", lambda b: tp.fp8_pack([b])), (r"X\[0\]", lambda b: tp.fp8_matmul([b], [XS], [W], [WSC])),
    (r"W\[0\]", lambda b: tp.fp8_matmul([X], [XS], [b], [WSC])),
    (r"A\[0\]", lambda b: tp.fp8_weight_grad([b], [XS], [X], [XS])),
    (r"B\[0\]", lambda b: tp.fp8_weight_grad([X], [XS], [b], [XS])), ("logits", lambda b: tp.expert_route(b, 2)),
    ("logits", lambda b: tp.expert_route_backward(ROUTE.weights, b, ROUTE)),
    (r"X\[0\]", lambda b: tp.expert_matmul([b], [XS], [W], [WSC], ROUTE)),
    ("rows", lambda b: tp.expert_combine(b, ROUTE)), ("rows", lambda b: tp.expert_combine_backward(X, b, ROUTE)),
])
def test_matrices_are_asked_for_by_name(name, call, bad, what):
    with pytest.raises(ValueError, match=name + " " + what):
        call(bad)


@pytest.mark.parametrize("call,what", [
    (lambda: tp.fp8_pack([]), "no shards"), (lambda: tp.fp8_pack([host(4, 64)]), "not on a GPU"),
    (lambda: tp.fp8_pack([host(4, 64)], rows=False), "neither rows nor columns"),
    (lambda: tp.fp8_pack([host(4, 64)], gather=True), "gather needs a route"),
    (lambda: tp.fp8_matmul([X], [XS, XS], [W], [WSC]), "x_scales: 2 tensors"),
    (lambda: tp.fp8_matmul([X], [XS], [W], [WSC]), "not on a GPU"),
    (lambda: tp.fp8_weight_grad([X], [XS], [X, X], [XS]), "B: 2 tensors"),
    (lambda: tp.expert_route(host(4, 8), 2, score="tanh"), "score must be"),
    (lambda: tp.expert_route(host(4, 8), 2), "not on a GPU"),
    (lambda: tp.expert_matmul([X], [XS], [W], [WSC], ROUTE), "not on a GPU"),
    (lambda: tp.expert_combine(host(8, 64), ROUTE), "not on a GPU"),
])
def test_other_arguments_are_refused(call, what):
    with pytest.raises(ValueError, match=what):
        call()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_oracle_gradient_against_differences(score, renorm):
    g = torch.Generator().manual_seed(3)
    x, dw = torch.randn(5, 9, generator=g, dtype=torch.float64), torch.randn(5, 3, generator=g, dtype=torch.float64)
    mask = torch.tensor([1, 1, 0, 1, 1], dtype=torch.bool)
    ids = O.choose(x, 3, score, None, 1, 1, mask)
    w = O.route_weights(x, ids, score, renorm, 1.7)
    d, _ = O.route_gradient(x, ids, w, dw, score, renorm, 1.7)
    h = 2.0 ** -20
    for e in range(9):
        up, down = x.clone(), x.clone()
        up[:, e] += h
        down[:, e] -= h
        slope = ((O.route_weights(up, ids, score, renorm, 1.7) - O.route_weights(down, ids, score, renorm, 1.7)) * dw).sum(1) / (2 * h)
        # the third derivative is below 10 |dw|: h^2 of it and 2^-52 / h of the quotient's rounding
        assert (slope - d[:, e]).abs().max() <= 10 * dw.abs().sum(1).max() * h * h + 2.0 ** -28


def test_tokens_are_counted_in_32_bits_to_the_end_of_the_last_part():
    for T, want in ((2 ** 31 - 1, SHAPE), (2 ** 31 - 2 ** 17, SHAPE), (2 ** 31 - 2 ** 17 - 1, INVALID)):     # the handle
        assert route(T=T, E=1, k=1, nb=1 << 40) == want
        assert rgrad(T=T, E=1, k=1) == want
