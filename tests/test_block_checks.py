"""Refusals of the MLP block's operators, and the oracle's gradients against
differences.  No GPU: the C ABI is called with a NULL handle and pointers that
are never followed (a check that passed would end at the NULL handle), the
binding with host tensors."""
import pytest
import torch

import block_oracle as O
from tensor_gemm_reduction_amd import tpfuse as tp

A, MIS8, MIS2, ODD = 0x1000, 0x1008, 0x1002, 0x1001
BF = torch.bfloat16


def arr(v, n=2):
    return tp.ptr_array(v if isinstance(v, list) else [v] * n)


def norm(p=2, M=4, H=64, x=A, xt=0, blocks=A, bt=0, wq=A, wp=A, gate=A, kind=1, wt=0, x_out=A, y=A, stats=None):
    return tp.load().tpf_block_norm(None, p, M, H, x, xt, arr(blocks) if blocks else None, bt, wq, wp, gate, kind, wt,
                                    1.0, 1.0, 1e-6, 0, x_out, y, stats, None)


def norm_bwd(p=2, M=4, H=64, dy=A, dxo=A, x=A, xt=0, blocks=A, bt=0, stats=A, wq=A, wp=A, gate=A, kind=1, wt=0, dx=A,
             db=A, dwq=A, dwp=A, dg=A, ws=A, nb=None):
    lib = tp.load()
    nb = lib.tpf_block_norm_backward_ws(M, H) if nb is None else nb
    return lib.tpf_block_norm_backward(None, p, M, H, dy, dxo, x, xt, arr(blocks), bt, stats, wq, wp, gate, kind, wt,
                                       1.0, 1.0, 0, dx, db, dwq, dwp, dg, ws, nb, None)


def pack(p=2, M=4, F=64, u=A, gelu=1, h=A, codes=A, scales=ODD):
    return tp.load().tpf_stash_pack(None, p, M, F, arr(u), gelu, arr(h) if h else None, arr(codes), arr(scales), None)


def bwd(p=2, M=4, F=64, codes=A, scales=ODD, dh=A, du=A, h=A):
    return tp.load().tpf_stash_backward(None, p, M, F, arr(codes), arr(scales), arr(dh), arr(du), arr(h), None)


def grad(p=2, M=4, R=64, C=32, codes=A, scales=ODD, dy=A, dw=A, dt=0):
    return tp.load().tpf_stash_weight_grad(None, p, M, R, C, arr(codes), arr(scales), arr(dy), arr(dw), dt, A, 1 << 40,
                                           None)


def qw(p=2, M=4, K=64, N=7, group=32, x=A, codes=A, scales=MIS2, zeros=ODD, y=A, yt=0):
    return tp.load().tpf_qweight_matmul(None, p, M, K, N, group, arr(x), arr(codes), arr(scales),
                                        arr(zeros) if zeros else None, 0, y, yt, A, 1 << 40, None)


INVALID, SHAPE, ALIGN, WS, UNSUP = (tp.ERR_INVALID_ARG, tp.ERR_SHAPE, tp.ERR_ALIGNMENT, tp.ERR_WORKSPACE,
                                    tp.ERR_UNSUPPORTED)


@pytest.mark.parametrize("call,kw,code", [
    (norm, dict(p=0), SHAPE), (norm, dict(p=17), SHAPE), (norm, dict(M=0), SHAPE), (norm, dict(H=-8), SHAPE),
    (norm, dict(M=1 << 31), SHAPE), (norm, dict(H=12), ALIGN), (norm, dict(H=32776), UNSUP), (norm, dict(xt=2), INVALID),
    (norm, dict(bt=-1), INVALID), (norm, dict(wt=5), INVALID), (norm, dict(kind=3), INVALID),
    (norm, dict(gate=None), INVALID), (norm, dict(x=None), INVALID), (norm, dict(x=MIS8), ALIGN),
    (norm, dict(blocks=None), INVALID), (norm, dict(blocks=[A, 0]), INVALID), (norm, dict(blocks=[A, MIS8]), ALIGN),
    (norm, dict(wq=None), INVALID), (norm, dict(wp=MIS2), ALIGN), (norm, dict(x_out=None), INVALID),
    (norm, dict(y=MIS8), ALIGN), (norm, dict(stats=MIS2), ALIGN),
    (norm_bwd, dict(H=20), ALIGN), (norm_bwd, dict(dy=None), INVALID), (norm_bwd, dict(dxo=MIS8), ALIGN),
    (norm_bwd, dict(stats=None), INVALID), (norm_bwd, dict(dg=None), INVALID), (norm_bwd, dict(dwq=MIS2), ALIGN),
    (norm_bwd, dict(ws=None), WS), (norm_bwd, dict(nb=100), WS), (norm_bwd, dict(ws=MIS8), ALIGN),
    (pack, dict(p=0), SHAPE), (pack, dict(M=0), SHAPE), (pack, dict(F=60), ALIGN), (pack, dict(u=[A, MIS8]), ALIGN),
    (pack, dict(h=None), INVALID), (pack, dict(codes=MIS2), ALIGN), (pack, dict(scales=[A, 0]), INVALID),
    (pack, dict(M=1 << 30, F=1 << 30), UNSUP),
    (bwd, dict(F=4), ALIGN), (bwd, dict(codes=[A, 0]), INVALID), (bwd, dict(dh=MIS8), ALIGN), (bwd, dict(du=[A, 0]), INVALID),
    (grad, dict(R=12), ALIGN), (grad, dict(C=4), ALIGN), (grad, dict(M=0), SHAPE), (grad, dict(dt=3), INVALID),
    (grad, dict(codes=MIS2), ALIGN), (grad, dict(dy=MIS8), ALIGN), (grad, dict(R=1 << 16, C=1 << 16), UNSUP),
    (qw, dict(group=16), UNSUP), (qw, dict(group=256, K=256), UNSUP), (qw, dict(K=96, group=64), SHAPE),
    (qw, dict(N=0), SHAPE), (qw, dict(x=MIS8), ALIGN), (qw, dict(codes=MIS8), ALIGN), (qw, dict(scales=ODD), ALIGN),
    (qw, dict(zeros=[A, 0]), INVALID), (qw, dict(y=None), INVALID), (qw, dict(yt=9), INVALID),
    (qw, dict(N=1 << 20, K=1 << 14), UNSUP),
])
def test_refusals(call, kw, code):
    assert call(**kw) == code
    assert tp.load().tpf_last_error()


@pytest.mark.parametrize("call,kw", [
    (norm, {}), (norm, dict(kind=0, gate=None)), (norm, dict(stats=0x1004)), (norm_bwd, {}), (norm_bwd, dict(dxo=None)),
    (norm_bwd, dict(kind=0, gate=None, dg=None)), (pack, {}), (pack, dict(gelu=0, h=None)), (pack, dict(codes=MIS8)),
    (bwd, {}), (bwd, dict(codes=MIS8)), (grad, {}), (grad, dict(codes=MIS8)), (qw, {}), (qw, dict(zeros=None)),
    (qw, dict(N=1, M=1))])
def test_good_arguments_reach_the_handle(call, kw):
    assert call(**kw) == INVALID
    assert tp.load().tpf_last_error() == b"handle is NULL"


def test_workspace_sizes():
    lib = tp.load()
    assert lib.tpf_block_norm_backward_ws(0, 64) == 0 and lib.tpf_block_norm_backward_ws(4, 12) == 0
    assert lib.tpf_block_norm_backward_ws(1, 64) == 2 * 64 * 4


def host(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


E4 = torch.float8_e4m3fn


@pytest.mark.parametrize("call", [
    lambda: tp.block_norm(host(4, 64), [host(4, 64)], host(64), host(64)),
    lambda: tp.block_norm_backward(host(4, 64), None, host(4, 64), [host(4, 64)], host(2, 4), host(64), host(64)),
    lambda: tp.stash_pack([host(4, 64)]),
    lambda: tp.stash_backward([host(4, 64, dtype=E4)], [host(1, 2, dtype=torch.uint8)], [host(4, 64)]),
    lambda: tp.stash_weight_grad([host(4, 64, dtype=E4)], [host(1, 2, dtype=torch.uint8)], [host(4, 32)]),
    lambda: tp.qweight_matmul([host(4, 64)], [host(8, 32, dtype=torch.uint8)], [host(8, 1)], group=64),
])
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="not on a GPU"):
        call()


@pytest.mark.parametrize("call,msg", [
    (lambda: tp.block_norm(host(4, 64), [], host(64), host(64)), "no tensors"),
    (lambda: tp.block_norm(host(64), [host(64)], host(64), host(64)), "dimensions"),
    (lambda: tp.stash_pack([]), "no shards"),
    (lambda: tp.stash_backward([host(4, 64, dtype=E4)] * 2, [host(1, 2, dtype=torch.uint8)], [host(4, 64)] * 2),
     "one per shard"),
    (lambda: tp.qweight_matmul([host(4, 96)], [host(8, 48, dtype=torch.uint8)], [host(8, 1)], group=64), "group"),
    (lambda: tp.qweight_matmul([host(4, 64)] * 2, [host(8, 32, dtype=torch.uint8)], [host(8, 1)] * 2, group=64),
     "one per shard"),
])
def test_counts_and_shapes_are_refused(call, msg):
    with pytest.raises(ValueError, match=msg):
        call()


@pytest.mark.gpu
def test_device_tensor_checks():
    def dev(*shape, dtype=BF):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    x, w, st = dev(4, 64), dev(64), dev(2, 4, dtype=torch.float32)
    u8 = torch.uint8
    for call, msg in [
        (lambda: tp.block_norm(x, [dev(4, 56)], w, w), "blocks has shape"),
        (lambda: tp.block_norm(x, [x, dev(4, 64, dtype=torch.float32)], w, w), "differ in dtype"),
        (lambda: tp.block_norm(x, [x], w, dev(64, dtype=torch.float32)), "w_post has dtype"),
        (lambda: tp.block_norm(x, [x], w, w, gate=dev(4, 2)), "gate has shape"),
        (lambda: tp.block_norm(dev(64, 4).t(), [x], w, w), "not contiguous"),
        (lambda: tp.block_norm(x, [x], w, w, x_out=dev(4, 64, dtype=torch.float32)), "x_out has dtype"),
        (lambda: tp.block_norm_backward(x, None, x, [x], dev(2, 5, dtype=torch.float32), w, w), "stats has shape"),
        (lambda: tp.block_norm_backward(x, None, x, [x], st, w, w, ws=dev(8, dtype=u8)), "workspace has 8 bytes"),
        (lambda: tp.stash_pack([dev(4, 64, dtype=torch.float32)]), "dtype"),
        (lambda: tp.stash_backward([dev(33, 64, dtype=E4)], [dev(1, 2, dtype=u8)], [dev(33, 64)]), "scales has shape"),
        (lambda: tp.stash_weight_grad([dev(4, 64, dtype=E4)], [dev(1, 2, dtype=u8)], [dev(5, 32)]), "dY has shape"),
        (lambda: tp.qweight_matmul([dev(4, 64)], [dev(8, 30, dtype=u8)], [dev(8, 1)], group=64), "codes has shape"),
        (lambda: tp.qweight_matmul([dev(4, 64)], [dev(8, 32, dtype=u8)], [dev(8, 2)], group=64), "scales has shape"),
    ]:
        with pytest.raises((ValueError, tp.TpfError), match=msg):
            call()


# --- the oracle itself ------------------------------------------------------

@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_oracle_norm_gradient_is_the_derivative(gate):
    """The backward's formula against the forward's differences (double precision)."""
    g = torch.Generator().manual_seed(0)
    M, H, p, alpha, beta, eps = 3, 8, 2, 0.8, 0.6, 1e-3

    def r(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    x, blocks, wq, wp = r(M, H), [r(M, H) for _ in range(p)], r(H), r(H)
    gt = None if gate is None else r(*((H,) if gate == "channel" else (M, 1)))
    dy, dxo = r(M, H), r(M, H)

    def loss(x, b0, wq, wp, gt):
        xo, _, _ = O.norm_forward(x, [b0, blocks[1]], wq, wp, gt, alpha, beta, eps, 1.0)
        return float((O.pre_norm(xo, wq, eps, 1.0)[0] * dy).sum() + (xo * dxo).sum())

    xo, _, rb = O.norm_forward(x, blocks, wq, wp, gt, alpha, beta, eps, 1.0)
    _, rx = O.pre_norm(xo, wq, eps, 1.0)
    got, _ = O.norm_backward(dy, dxo, xo, blocks, torch.stack([rb[:, 0], rx[:, 0]]), wq, wp, gt, alpha, beta, 1.0)
    args = [x, blocks[0], wq, wp, gt]
    d = 1e-5
    for i, name in enumerate(("dx", "db", "dw_pre", "dw_post", "dgate")):
        if args[i] is None:
            continue
        num = torch.zeros_like(args[i])
        for j in range(num.numel()):
            lo, hi = [a if a is None else a.clone() for a in args], [a if a is None else a.clone() for a in args]
            lo[i].view(-1)[j] -= d
            hi[i].view(-1)[j] += d
            num.view(-1)[j] = (loss(*hi) - loss(*lo)) / (2 * d)
        assert torch.allclose(got[name], num, rtol=1e-6, atol=1e-7), name


def test_oracle_gelu_gradient_is_the_derivative():
    u = torch.linspace(-9, 9, 2001, dtype=torch.float64)
    d = 1e-5
    num = ((u + d) * O.cdf(u + d) - (u - d) * O.cdf(u - d)) / (2 * d)
    assert torch.allclose(O.cdf(u) + u * O.pdf(u), num, atol=1e-9)


def test_oracle_pack_holds_known_codes():
    """Hand-worked: a block whose largest value is 448 keeps factor 1; 449 takes the next."""
    u = torch.zeros(32, 64)
    u[0, :5] = torch.tensor([448.0, 1.0, 17.0, 19.0, 0.001])
    u[0, 32] = 449.0
    codes, scales = O.pack(u)
    assert scales.tolist() == [[127, 128]]
    assert codes[0, :5].tolist() == [448.0, 1.0, 16.0, 20.0, 2.0 ** -9 * 0.0 + 0.001953125 * round(0.001 / 0.001953125)]
    assert codes[0, 32].item() == 224.0
    q, size = O.dequantize(torch.tensor([[0x21, 0x43, 0x65, 0x87] * 4], dtype=torch.uint8), torch.ones(1, 1), None, 32)
    assert q[0, :8].tolist() == [1 - 8, 3 - 8, 5 - 8, 7 - 8, 2 - 8, 4 - 8, 6 - 8, 8 - 8]
