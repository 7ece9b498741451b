"""The MLP block's operators on the sizes of production calls: the weight
gradient's large tiles, rounds of scales and cut contractions, and the norm
backward's column sums over many rows and workgroups."""
import pytest
import torch

import block_oracle as O
from test_gpu_block import BF, F32, D, ROUNDINGS
from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu

GRADS = [  # p, M, R, C
    (4, 200, 1800, 1544),       # 224 tiles of 256 x 256, ragged in every direction
    (13, 95, 1000, 1032),       # 260
    (1, 65, 3592, 3592),        # 225, one step and a row
    (2, 1, 2504, 2568),         # 220, one row
    (3, 513, 2048, 2048),       # 192: the fewest
    (2, 32900, 2504, 2568),     # 515 steps: two rounds of scales
    (1, 140001, 1024, 2048),    # four parts of 547 steps on 128 x 128 tiles
    (1, 4100, 64, 64),          # 16 parts
    (2, 1003, 328, 600),        # four parts
    (1, 1027, 136, 264),        # four parts, the last one ragged
]


@pytest.mark.parametrize("out", [F32, BF])
@pytest.mark.parametrize("p,M,R,C", GRADS)
def test_weight_gradient_of_whole_numbers(p, M, R, C, out):
    """Small whole numbers: every fp32 sum is exact in any order, so a row lost or doubled shows."""
    g = torch.Generator(device="cuda").manual_seed(M + R)
    u = [torch.randint(-4, 5, (M, R), generator=g, device="cuda").to(BF) for _ in range(p)]
    y = [torch.randint(-3, 4, (M, C), generator=g, device="cuda").to(BF) for _ in range(p)]
    _, codes, scales = tp.stash_pack(u, gelu=False)
    dw = tp.stash_weight_grad(codes, scales, y, out_dtype=out)
    for k in range(p):
        want = u[k].to(D).t().contiguous() @ y[k].to(D)
        assert torch.equal(dw[k], want.to(out)), f"shard {k}: {int((dw[k] != want.to(out)).sum())} elements differ"


def test_weight_gradient_of_different_scales():
    """Blocks whose factors differ, whole numbers times them: exact as well."""
    g = torch.Generator(device="cuda").manual_seed(5)
    p, M, R, C = 4, 170, 1800, 1544
    power = torch.randint(0, 4, (p, -(-M // 32), -(-R // 32)), generator=g, device="cuda")
    power = power.repeat_interleave(32, 1).repeat_interleave(32, 2)[:, :M, :R]
    u = (torch.randint(-4, 5, (p, M, R), generator=g, device="cuda") * 2.0 ** power).to(BF)
    y = torch.randint(-3, 4, (p, M, C), generator=g, device="cuda").to(BF)
    _, codes, scales = tp.stash_pack(u.unbind(0), gelu=False)
    assert len(torch.unique(torch.stack(scales))) >= 4
    dw = tp.stash_weight_grad(codes, scales, y.unbind(0))
    for k in range(p):
        assert torch.equal(dw[k], (u[k].to(D).t().contiguous() @ y[k].to(D)).to(F32))


COLUMNS = [  # M, H, x, blocks, gate, vectors
    (8192, 64, BF, BF, "channel", BF),          # 1024 workgroups of eight rows
    (40001, 64, F32, BF, "token", F32),         # 4096 workgroups, nine or ten rows each
    (5000, 1032, BF, F32, "channel", F32),
    (700, 8192, F32, F32, "channel", F32),      # 256 workgroups, two or three rows
    (700, 8200, BF, BF, "token", BF),           # rows of two vectors a thread
    (600, 16384, F32, BF, "channel", F32),
    (520, 16392, BF, F32, "channel", BF),       # rows of four
    (400, 32768, F32, F32, "token", F32),
    (400, 32768, BF, BF, "channel", BF),
]


@pytest.mark.parametrize("M,H,xt,bt,gate,vt", COLUMNS)
def test_norm_column_sums(M, H, xt, bt, gate, vt):
    g = torch.Generator(device="cuda").manual_seed(M + H)

    def rand(*s, std=1.0, dtype=F32):
        return (torch.randn(s, device="cuda", generator=g) * std).to(dtype)

    x, b = rand(M, H, std=2.0, dtype=xt), rand(M, H, std=0.7, dtype=bt)
    wq, wp = (1 + rand(H, std=0.2)).to(vt), (1 + rand(H, std=0.2)).to(vt)
    gt = (0.5 + rand(*((H,) if gate == "channel" else (M, 1)), std=0.3)).to(vt)
    dy, dxo = rand(M, H, std=0.5, dtype=BF), rand(M, H, std=0.5, dtype=xt)
    stats = torch.stack([(t.to(D).square().mean(1) + 1e-6).rsqrt().float() for t in (b, x)])
    got = dict(zip(("dx", "db", "dw_pre", "dw_post", "dgate"),
                   tp.block_norm_backward(dy, dxo, x, [b], stats, wq, wp, gt, alpha=1.1, beta=0.6)))
    want, size = O.norm_backward(dy, dxo, x, [b], stats, wq, wp, gt, 1.1, 0.6, 0.0)
    for name, w in want.items():
        # a row's terms; for the sums down the columns also the rows of a workgroup (at most ten), then 64 strips of
        # workgroups (at most 64 each) in two joins of eight
        down = 0 if name in ("dx", "db") or (name == "dgate" and gate == "token") else 10 + 64 + 16
        bound = (2 * ROUNDINGS + down * O.STEP) * size[name]
        t = got[name].dtype
        bad = (got[name].to(D) - w).abs() > bound + (O.half_step(t) if t is BF else O.STEP) * w.abs()
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} out"


def shifted(t, by):
    """A copy of `t` whose address is `by` bytes past a multiple of 256."""
    n = t.numel() * t.element_size()
    buf = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    buf[by:by + n] = t.contiguous().view(torch.uint8).view(-1)
    v = buf[by:by + n].view(t.dtype).view(t.shape)
    assert v.data_ptr() % 256 == by
    return v


def test_least_alignments():
    """Codes at odd multiples of 8 bytes, scales at odd addresses (of 2 bytes for the 4-bit weights)."""
    g = torch.Generator(device="cuda").manual_seed(2)
    u = torch.randn(100, 264, device="cuda", generator=g).to(BF)
    dy = torch.randn(100, 264, device="cuda", generator=g).to(BF)
    _, (codes,), (scales,) = tp.stash_pack([u], gelu=False)
    at8, odd = shifted(codes.view(torch.uint8), 8), shifted(scales, 7)
    for a, b in zip(tp.stash_backward([codes], [scales], [dy]), tp.stash_backward([at8], [odd], [dy])):
        assert torch.equal(a[0], b[0])
    assert torch.equal(tp.stash_weight_grad([codes], [scales], [dy])[0], tp.stash_weight_grad([at8], [odd], [dy])[0])
    for M, K, N, group in ((3, 160, 70, 32), (40, 384, 200, 128)):
        x = torch.randn(M, K, device="cuda", generator=g).to(BF)
        q = torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
        s = torch.rand(N, K // group, device="cuda", generator=g).to(BF)
        z = torch.randint(0, 16, (N, K // group), device="cuda", generator=g, dtype=torch.uint8)
        want = tp.qweight_matmul([x], [q], [s], [z], group=group)
        assert torch.equal(want, tp.qweight_matmul([x], [q], [shifted(s, 6)], [shifted(z, 3)], group=group))
