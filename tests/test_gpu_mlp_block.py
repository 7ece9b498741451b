"""The MLP block on the library's calls, against the same block in float64 on
the CPU with the bf16 tensors that pass between its steps rounded alike."""
import pytest
import torch

import block_oracle as O
from tensor_gemm_reduction_amd import mlp_block as mb

D = torch.float64


def rms(a):
    return float(a.to(D).square().mean().sqrt())


def test_quantize_keeps_each_weight_within_half_a_step():
    g = torch.Generator().manual_seed(1)
    for N, K, group in ((5, 64, 32), (16, 256, 64), (3, 384, 128)):
        w = torch.randn(N, K, generator=g).bfloat16()
        codes, scales, zeros = mb.quantize(w, group)
        back, _ = O.dequantize(codes, scales, zeros, group)
        step = torch.repeat_interleave(scales.to(D), group, 1)
        # half a step for the code, half for the rounded zero point; the scale's own rounding
        # (2^-8) can cost the extremes 15 steps 2^-8
        assert ((back - w.to(D)).abs() <= (1.0 + 15 * 2.0 ** -8) * step).all()


def block_and_inputs(p=2, M=96, H=256, F=128):
    g = torch.Generator().manual_seed(7)

    def rand(*s, std=1.0):
        return torch.randn(s, generator=g) * std

    W1 = [rand(H, F, std=H ** -0.5).bfloat16() for _ in range(p)]
    W2 = [rand(F, H, std=F ** -0.5).bfloat16() for _ in range(p)]
    vec = [1 + rand(H, std=0.1) for _ in range(3)]
    x, y, dy, dx = rand(M, H).bfloat16(), rand(M, H).bfloat16(), rand(M, H, std=0.1).bfloat16(), rand(M, H, std=0.1).bfloat16()
    return W1, W2, vec, x, y, dy, dx


@pytest.mark.gpu
def test_training_step():
    W1, W2, (wq, wp, gate), x, y, dy, dxo = block_and_inputs()
    blk = mb.MLPBlock([w.cuda() for w in W1], [w.cuda() for w in W2], wq.cuda(), wp.cuda(), gate.cuda(), beta=0.5)
    x_out, y_next, kept = blk.forward(x.cuda(), y.cuda())
    grads = blk.backward(dy.cuda(), dxo.cuda(), kept)

    # the same block by autograd in double precision
    leaves = [t.to(D).requires_grad_() for t in (x, y, wq, wp, gate, *W1, *W2)]
    lx, ly, lq, lp, lg = leaves[:5]
    l1, l2 = leaves[5:5 + len(W1)], leaves[5 + len(W1):]
    u = [ly @ w for w in l1]
    b = sum((t * O.cdf(t)) @ w for t, w in zip(u, l2))
    xo = lx + 0.5 * lg * lp * b * (b.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    yn = xo * (xo.square().mean(1, keepdim=True) + 1e-6).rsqrt() * lq
    torch.autograd.backward([xo, yn], [dxo.to(D), dy.to(D)])
    # Forward: u, h and b are rounded to bf16 (2^-9 rms each, h also carries u's), then the result.
    for got, want in ((x_out, xo.detach()), (y_next, yn.detach())):
        assert rms(got.cpu().to(D) - want) <= 6 * 2.0 ** -9 * rms(want)
    # Backward: the 8-bit activations are off by up to 2^-4 of themselves, 2^-5 rms, which enters every
    # gradient that passes through them once (W1, W2) or through GeLU's slope (W1, y); the rest carry only
    # bf16 roundings.
    loose = 2 * 2.0 ** -5
    for name, got, want, tol in (
            ("x", grads["x"], lx.grad, 8 * 2.0 ** -9), ("w_pre", grads["w_pre"], lq.grad, 8 * 2.0 ** -9),
            ("w_post", grads["w_post"], lp.grad, 16 * 2.0 ** -9), ("gate", grads["gate"], lg.grad, 16 * 2.0 ** -9),
            ("y", grads["y"], ly.grad, loose), ("W1", torch.stack(grads["W1"]), torch.stack([t.grad for t in l1]), loose),
            ("W2", torch.stack(grads["W2"]), torch.stack([t.grad for t in l2]), loose)):
        assert rms(got.cpu().to(D) - want) <= tol * rms(want), name


@pytest.mark.gpu
def test_decode_step():
    W1, W2, (wq, wp, gate), x, y, _, _ = block_and_inputs(M=3)
    blk = mb.MLPBlock([w.cuda() for w in W1], [w.cuda() for w in W2], wq.cuda(), wp.cuda(), gate.cuda())
    q = mb.QuantMLPBlock(blk, group=64)
    W1q = [O.dequantize(*(t.cpu() for t in w), 64)[0] for w in q.W1]
    W2q = [O.dequantize(c.cpu(), s.cpu(), z.cpu(), 64)[0] for c, s, z in zip(*q.W2)]
    u = [y.to(D) @ w.t() for w in W1q]
    b = sum((t * O.cdf(t)).bfloat16().to(D) @ w.t() for t, w in zip(u, W2q))
    want, _, _ = O.norm_forward(x, [b], wq, wp, gate, 1.0, 1.0, 1e-6, 0.0)
    xd = x.cuda()
    x_out, y_next = q.step(xd, y.cuda())
    assert x_out is xd
    assert rms(x_out.cpu().to(D) - want) <= 3 * 2.0 ** -9 * rms(want)
    wy, _ = O.pre_norm(x_out.cpu(), wq, 1e-6, 0.0)
    assert rms(y_next.cpu().to(D) - wy) <= 2 * 2.0 ** -9 * rms(wy)


@pytest.mark.gpu
def test_example_learns():
    losses = mb.example(tokens=128, H=256, F=128, p=2, steps=4)
    assert losses[-1] < losses[0]
