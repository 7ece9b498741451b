"""Every combination of types and row lengths that has a kernel of its own: the
norms in both directions, and 4-bit products of 33 and more rows."""
import pytest
import torch

import block_oracle as O
from test_gpu_block import BF, F32, D, ROUNDINGS, frame, qweight_case
from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu
TYPES = [(xt, bt, vt) for xt in (BF, F32) for bt in (BF, F32) for vt in (BF, F32)]
NAMES = ("dx", "db", "dw_pre", "dw_post", "dgate")


def operands(M, H, xt, bt, vt, gate, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s, std=1.0, mean=0.0, dtype=F32):
        return (mean + torch.randn(s, device="cuda", generator=g) * std).to(dtype)

    return dict(x=normal(M, H, std=2.0, dtype=xt), block=normal(M, H, std=0.7, dtype=bt),
                w_pre=normal(H, std=0.2, mean=1.0, dtype=vt), w_post=normal(H, std=0.2, mean=1.0, dtype=vt),
                gate=normal(*((H,) if gate == "channel" else (M, 1)), std=0.3, mean=0.5, dtype=vt),
                dy=normal(M, H, std=0.5, dtype=BF), dx_out=normal(M, H, std=0.5, dtype=xt))


def both(c, alpha=0.9, beta=0.6):
    kw = dict(w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"], alpha=alpha, beta=beta)
    x_out, y, stats = tp.block_norm(c["x"], [c["block"]], want_stats=True, **kw)
    return x_out, y, stats, dict(zip(NAMES, tp.block_norm_backward(c["dy"], c["dx_out"], x_out, [c["block"]], stats, **kw)))


@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("H", [1032, 12296, 20488])
@pytest.mark.parametrize("xt,bt,vt", TYPES)
def test_norm(xt, bt, vt, H, gate):
    M = 7
    c = operands(M, H, xt, bt, vt, gate, seed=H)
    x_out, y, stats, got = both(c)

    def near(t, want, size, what):
        bad = (t.to(D) - want).abs() > size + (O.half_step(t.dtype) if t.dtype is BF else O.STEP) * want.abs()
        assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out"

    want, size, rb = O.norm_forward(c["x"], [c["block"]], c["w_pre"], c["w_post"], c["gate"], 0.9, 0.6, 1e-6, 0.0)
    near(x_out, want, (ROUNDINGS + O.STEP) * size, "x_out")
    wy, rx = O.pre_norm(x_out, c["w_pre"], 1e-6, 0.0)
    near(y, wy, ROUNDINGS * wy.abs(), "y")
    for i, w in enumerate((rb, rx)):
        near(stats[i], w[:, 0], ROUNDINGS * w[:, 0], "stats")
    grads, sizes = O.norm_backward(c["dy"], c["dx_out"], x_out, [c["block"]], stats, c["w_pre"], c["w_post"], c["gate"],
                                   0.9, 0.6, 0.0)
    for name, w in grads.items():
        near(got[name], w, (2 * ROUNDINGS + M * O.STEP) * sizes[name], name)


@pytest.mark.parametrize("H", [8192, 16384, 32768])
@pytest.mark.parametrize("xt,bt,vt", TYPES)
def test_norm_outputs_past_the_caches_are_those_of_small_calls(xt, bt, vt, H):
    M = (1 << 28) // (H * (4 if xt is BF else 6)) + 5
    c = operands(M, H, xt, bt, vt, "channel", seed=M)
    x_out, y, stats, got = both(c)
    for r in (slice(0, 6), slice(M - 6, M)):
        part = {k: v[r].contiguous() if v.dim() == 2 else v for k, v in c.items()}
        px, py, ps, pg = both(part)
        assert torch.equal(x_out[r], px) and torch.equal(y[r], py) and torch.equal(stats[:, r], ps)
        assert torch.equal(got["dx"][r], pg["dx"]) and torch.equal(got["db"][r], pg["db"])


@pytest.mark.parametrize("p,M,K,N,zeros", [(1, 33, 64, 128, True), (2, 64, 192, 200, True), (3, 50, 1088, 131, False),
                                           (1, 130, 320, 260, True), (8, 64, 896, 384, True)])
@pytest.mark.parametrize("out", [F32, BF])
def test_qweight_groups_of_64(p, M, K, N, zeros, out):
    c = qweight_case(p, M, K, N, 64, zeros, seed=3)
    y = tp.qweight_matmul(frame(c["x"]), frame(c["codes"]), frame(c["scales"]), frame(c["zeros"]) if zeros else None,
                          group=64, out_dtype=out).cpu().to(D)
    want, size = torch.zeros(M, N, dtype=D), torch.zeros(M, N, dtype=D)
    for k in range(p):
        w, wa = O.dequantize(c["codes"][k], c["scales"][k], c["zeros"][k] if zeros else None, 64)
        want += c["x"][k].to(D) @ w.t()
        size += c["x"][k].to(D).abs() @ wa.t()
    # a group's sums round once a product at most, the joining once a group
    bound = (64 + p * K / 64 + 16) * O.STEP * size
    assert ((y - want).abs() <= bound + (O.half_step(BF) * want.abs() if out is BF else 0)).all()


@pytest.mark.parametrize("M,N", [(20, 200), (64, 200)])
def test_qweight_whole_numbers_in_groups_of_64(M, N):
    """Whole numbers with a power of two for a scale: exact in any order."""
    c = qweight_case(2, M, 1152, N, 64, True, seed=4)
    g = torch.Generator().manual_seed(M)
    x = [torch.randint(-8, 9, (M, 1152), generator=g).to(BF) for _ in range(2)]
    s = [torch.full((N, 18), 0.25).to(BF) for _ in range(2)]
    y = tp.qweight_matmul(frame(x), frame(c["codes"]), frame(s), frame(c["zeros"]), group=64, out_dtype=F32)
    want = sum(x[k].to(D) @ O.dequantize(c["codes"][k], s[k], c["zeros"][k], 64)[0].t() for k in range(2))
    assert torch.equal(y.cpu().to(D), want)
