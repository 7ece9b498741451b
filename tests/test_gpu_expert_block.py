"""The MLP block of experts on the library's calls, against the same block in
float64 on the CPU: weights as their codes stand for them, everything else exact."""
import pytest
import torch

import block_oracle as BO
import scaled_oracle as O
from tensor_gemm_reduction_amd import expert_block as eb

D = torch.float64
E8 = 2.0 ** -5              # the rounding of e4m3: up to 2^-4 of the value, about half of that rms


def rms(a):
    return float(a.to(D).square().mean().sqrt())


def shape_of(w):
    return w.shape[:-2] + (O.blocks(w.shape[-2]), O.blocks(w.shape[-1]))


@pytest.mark.parametrize("shape", [(8, 16), (128, 128), (130, 272), (3, 256, 144)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize(shape, dtype):
    g = torch.Generator().manual_seed(5)
    w = (torch.randn(shape, generator=g) * torch.exp2(torch.randint(-20, 20, shape, generator=g).float())).to(dtype)
    w[..., :128, :128] = 0.0
    w[..., 0, 0] = 448.0 * 2.0 ** -3          # e4m3's largest at a power of two
    if shape[-1] > 128:
        w[..., :128, 128:256] = 0.0           # a block of zeros
    codes, scales = eb.quantize(w)
    assert scales.shape == shape_of(w) and scales.dtype == torch.uint8 and codes.shape == w.shape
    flat = lambda t: t.reshape((-1,) + t.shape[-2:])
    for c, s, v in zip(flat(codes.view(torch.uint8)), flat(scales), flat(w)):
        back, step = O.weight(c.view(torch.float8_e4m3fn), s), O.weight(torch.ones(v.shape).to(torch.float8_e4m3fn), s)
        # half a step of e4m3, and of its least numbers, 2^-9
        assert ((back - v.to(D)).abs() <= (v.to(D).abs() * 2.0 ** -4).clamp(min=2.0 ** -10 * step)).all()
        assert int(s[0, 0]) == 124
        top = torch.zeros(s.shape, dtype=D)
        for i in range(s.shape[0]):
            for j in range(s.shape[1]):
                top[i, j] = v[128 * i:128 * i + 128, 128 * j:128 * j + 128].to(D).abs().max()
        least = torch.exp2(s.to(D) - 127)
        assert (top <= 448 * least).all() and ((top > 224 * least) | (s == 10)).all()
    t, ts = eb._turned(codes, scales)
    assert torch.equal(t.view(torch.uint8), codes.view(torch.uint8).transpose(-1, -2))
    assert torch.equal(ts, scales.transpose(-1, -2)) and t.is_contiguous() and ts.is_contiguous()


def block_and_inputs(T, shared, p=2, H=256, F=128, E=8, k=3, **how):
    g = torch.Generator().manual_seed(11)

    def rand(*s, std=1.0):
        return torch.randn(s, generator=g) * std

    def shards(*s, std):
        return [rand(*s, std=std).bfloat16().cuda() for _ in range(p)]

    vec = [(1 + rand(H, std=0.1)).cuda() for _ in range(3)]
    more = dict(V1=shards(F + 16, H, std=H ** -0.5), V2=shards(H, F + 16, std=F ** -0.5)) if shared else {}
    blk = eb.ExpertBlock(rand(H, E, std=H ** -0.5).bfloat16().cuda(), shards(E, F, H, std=H ** -0.5),
                         shards(E, H, F, std=F ** -0.5), k, *vec, beta=0.5, **more, **how)
    return blk, rand(T, H).bfloat16(), rand(T, H).bfloat16(), rand(T, H, std=0.1).bfloat16(), rand(T, H, std=0.1).bfloat16()


def values(w):
    """Shards of a weight (of one or of each expert) as the codes stand for them."""
    out = []
    for c, s in zip(*w):
        c, s = c.cpu(), s.cpu()
        out.append(O.weight(c, s) if c.dim() == 2 else torch.stack([O.weight(a, b) for a, b in zip(c, s)]))
    return out


def exact(blk, x, y, mask, ids):
    """(leaves by name, x_out, y_next) of the block by definition; the experts are given."""
    leaves = {"x": x.to(D), "y": y.to(D), "Wr": blk.Wr.cpu().to(D)}
    leaves.update({n: blk.norm[n].cpu().to(D) for n in ("w_pre", "w_post", "gate")})
    lists = {"W1": values(blk.experts.w1), "W2": values(blk.experts.w2)}
    if blk.shared:
        lists.update(V1=values(blk.shared.w1), V2=values(blk.shared.w2))
    leaves = {n: t.requires_grad_() for n, t in leaves.items()}
    lists = {n: [t.requires_grad_() for t in v] for n, v in lists.items()}
    gelu = lambda t: t * BO.cdf(t)
    score = blk.weighing["score"]
    logits = leaves["y"] @ leaves["Wr"]
    s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    routed = ids[:, 0] >= 0
    w = torch.gather(s, 1, ids.clamp(min=0).long())
    w = w / w.sum(1, keepdim=True) * blk.weighing["scale"] * routed[:, None]
    b = torch.zeros_like(leaves["x"])
    for e in range(blk.Wr.shape[1]):
        rows = sum(gelu(leaves["y"] @ a[e].t()) @ c[e].t() for a, c in zip(lists["W1"], lists["W2"]))
        b = b + rows * torch.where(ids == e, w, 0.0).sum(1, keepdim=True)
    if blk.shared:
        b = b + sum(gelu(leaves["y"] @ a.t()) @ c.t() for a, c in zip(lists["V1"], lists["V2"]))
    norm = lambda t: t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    xo = leaves["x"] + 0.5 * leaves["gate"] * leaves["w_post"] * norm(b)
    return leaves, lists, xo, norm(xo) * leaves["w_pre"]


@pytest.mark.gpu
@pytest.mark.parametrize("T,shared,masked,how", [
    (96, False, False, {}), (200, True, True, dict(score="sigmoid", scale=2.5)), (333, True, False, dict(groups=4, top_groups=2))])
def test_training_step(T, shared, masked, how):
    blk, x, y, dy, dxo = block_and_inputs(T, shared, **how)
    mask = torch.arange(T) % 5 != 2 if masked else None
    x_out, y_next, kept = blk.forward(x.cuda(), y.cuda(), mask.cuda() if masked else None)
    grads = blk.backward(dy.cuda(), dxo.cuda(), kept)
    ids = kept[2].ids.cpu()
    if masked:
        assert torch.equal(ids[:, 0] >= 0, mask)
    leaves, lists, xo, yn = exact(blk, x, y, mask, ids)
    torch.autograd.backward([xo, yn], [dxo.to(D), dy.to(D)])
    # Roundings of one size E8 each, rms, that are independent.  b: y's and h's (and GeLU's slope on the
    # first, up to 1.3): 2, of which x_out and y_next carry less.
    for got, want in ((x_out, xo.detach()), (y_next, yn.detach())):
        assert rms(got.cpu().to(D) - want) <= 2 * E8 * rms(want)
    # The norm's gradients carry b's 2.  The experts' rows' carry them twice (the norm's statistics and its
    # direction) and their own: 3; with h from u's codes W2's is 4; W1's has u's codes once more in the slope,
    # its own and y's rounding: 5; y's, W1's without y's, through the weights' gradients as well: 5.  Those
    # are differences of rows' products with db (3 each), twice their own size at most.
    tol = {"x": 2, "w_pre": 2, "w_post": 3, "gate": 3, "W2": 4, "V2": 4, "W1": 5, "V1": 5, "y": 5, "Wr": 8}
    for name, t in leaves.items():
        assert rms(grads[name].cpu().to(D) - t.grad) <= tol[name] * E8 * rms(t.grad), name
    for name, v in lists.items():
        got, want = torch.stack(grads[name]).cpu(), torch.stack([t.grad for t in v])
        assert rms(got.to(D) - want) <= tol[name] * E8 * rms(want), name


@pytest.mark.gpu
@pytest.mark.parametrize("T,shared,masked", [(1, True, False), (3, False, False), (16, True, True)])
def test_decode_step(T, shared, masked):
    blk, x, y, _, _ = block_and_inputs(T, shared)
    mask = torch.arange(T) % 2 == 0 if masked else None
    dmask = mask.cuda() if masked else None
    _, route = blk.route(y.cuda(), dmask)
    _, _, xo, yn = exact(blk, x, y, mask, route.ids.cpu())
    xd = x.cuda()
    x_out, y_next = blk.step(xd, y.cuda(), dmask)
    assert x_out is xd
    for got, want in ((x_out, xo.detach()), (y_next, yn.detach())):
        assert rms(got.cpu().to(D) - want) <= 2 * E8 * rms(want)


@pytest.mark.gpu
def test_example_runs():
    losses = eb.example(tokens=160, H=256, F=128, E=8, k=2, p=2, steps=2)
    assert len(losses) == 2 and all(0 < v < 1e3 for v in losses)
