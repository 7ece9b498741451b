"""The MLP block's operators where a size chooses another path: outputs stored
past the caches, 4-bit products whose units cross shards, cut contractions."""
import pytest
import torch

import block_oracle as O
from test_gpu_block import BF, F32, D, close, frame, qweight_case
from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu


def noise(*shape, std=1.0, dtype=BF, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


@pytest.mark.parametrize("M,H,xt", [(8200, 8192, BF), (2760, 16384, F32)])
def test_large_norm_rows_are_those_of_small_calls(M, H, xt):
    """A row's results do not depend on how many rows there are, nor on how they are stored."""
    x, b = noise(M, H, std=2.0, dtype=xt), noise(M, H, seed=1)
    w, g = noise(H, dtype=F32, seed=2), noise(H, dtype=F32, seed=3)
    x_out, y, st = tp.block_norm(x, [b], w, w, g, alpha=0.9, beta=0.5, want_stats=True)
    dy, dxo = noise(M, H, seed=4), noise(M, H, dtype=xt, seed=5)
    dx, db, *_ = tp.block_norm_backward(dy, dxo, x_out, [b], st, w, w, g, alpha=0.9, beta=0.5)
    for r in (slice(0, 40), slice(M - 33, M)):
        part = tp.block_norm(x[r].contiguous(), [b[r].contiguous()], w, w, g, alpha=0.9, beta=0.5, want_stats=True)
        for got, want in zip((x_out[r], y[r], st[:, r]), part):
            assert torch.equal(got, want)
        back = tp.block_norm_backward(dy[r].contiguous(), dxo[r].contiguous(), part[0], [b[r].contiguous()], part[2],
                                      w, w, g, alpha=0.9, beta=0.5)
        assert torch.equal(dx[r], back[0]) and torch.equal(db[r], back[1])


def test_large_stash_rows_are_those_of_small_calls():
    p, M, F = 2, 8192, 8200                     # act: 269 MB, du and act: 537 MB
    u = [noise(M, F, std=3.0, seed=k) for k in range(p)]
    h, codes, scales = tp.stash_pack(u)
    dh = [noise(M, F, std=0.1, seed=9 + k) for k in range(p)]
    du, act = tp.stash_backward(codes, scales, dh)
    for r in (slice(0, 64), slice(M - 32, M)):
        blocks = slice(r.start // 32, r.stop // 32)
        part = tp.stash_pack([t[r].contiguous() for t in u])
        back = tp.stash_backward(part[1], part[2], [t[r].contiguous() for t in dh])
        for k in range(p):
            assert torch.equal(h[k][r], part[0][k])
            assert torch.equal(codes[k][r].view(torch.uint8), part[1][k].view(torch.uint8))
            assert torch.equal(scales[k][blocks], part[2][k])
            assert torch.equal(du[k][r], back[0][k]) and torch.equal(act[k][r], back[1][k])


CASES = [  # p, M, K, N, group, zeros, gelu
    (16, 1, 32, 40, 32, True, False),         # four shards in one block of units
    (5, 7, 96, 4100, 32, False, False),       # blocks across shards, 32 columns a workgroup
    (3, 16, 640, 4112, 128, True, True),      # five units a shard: blocks of four straddle
    (1, 2, 128, 5000, 64, False, False),      # fewer units than waves
    (7, 17, 64, 33, 64, True, False),         # the kernel for more rows, one unit a shard
    (2, 33, 2048, 131, 32, False, True),      # cut contraction, an output not in fours
    (4, 64, 1152, 384, 128, True, False),     # cut contraction whose parts end inside a shard
    (3, 32, 1312, 129, 32, True, False),      # a row's last unit of one run, a column alone in its workgroup
]


@pytest.mark.parametrize("p,M,K,N,group,zeros,gelu", CASES)
@pytest.mark.parametrize("out", [F32, BF])
def test_qweight_paths(p, M, K, N, group, zeros, gelu, out):
    c = qweight_case(p, M, K, N, group, zeros, seed=5)
    args = (frame(c["x"]), frame(c["codes"]), frame(c["scales"]), frame(c["zeros"]) if zeros else None)
    y = tp.qweight_matmul(*args, group=group, gelu=gelu, out_dtype=out)
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
    assert torch.equal(tp.qweight_matmul(*args, group=group, gelu=gelu, out_dtype=out), y)


def test_qweight_infinities_stay_in_their_row():
    """A row with an infinity or a NaN leaves the other rows' bits alone, also at a row's ragged end."""
    for M in (5, 40):
        c = qweight_case(2, M, 160, 70, 32, True, seed=2)
        args = [t.cuda() for t in c["codes"]], [t.cuda() for t in c["scales"]], [t.cuda() for t in c["zeros"]]
        x = [t.cuda() for t in c["x"]]
        want = tp.qweight_matmul(x, *args, group=32)
        x[0][1, 3], x[1][3, 159] = float("inf"), float("nan")
        got = tp.qweight_matmul(x, *args, group=32)
        keep = [r for r in range(M) if r not in (1, 3)]
        assert torch.equal(got[keep], want[keep])
        assert not got[1].isfinite().any() and got[3].isnan().all()
