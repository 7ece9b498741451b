"""The MLP block's operators with as many rows as a call accepts: row numbers
that, with a second index added, pass 31 bits, and grids of more threads than
one launch holds."""
import pytest
import torch

from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu
M, H = 2 ** 31 - 1, 8
BF = torch.bfloat16
# The rows that hold values: both ends, both sides of multiples of 2^28 rows (a launch's share) and of 2^30.
ROWS = sorted({r for c in (0, 1 << 28, 1 << 29, 3 << 28, 1 << 30, 5 << 28, 7 << 28, M - 1 - (M - 1) % 32)
               for r in range(max(0, c - 40), min(M, c + 72))})


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 200 GiB of GPU memory")
    yield
    torch.cuda.empty_cache()


def sparse(at, seed):
    """[M, H] of zeros but for the rows `at`, and those rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = torch.randn(len(at), H, device="cuda", generator=g).to(BF)
    t = torch.zeros(M, H, device="cuda", dtype=BF)
    t[at] = rows
    return t, rows


def same(t, at, rows, rest=0):
    """`t` holds `rows` at `at`, and `rest` elsewhere."""
    assert torch.equal(t[at], rows)
    t[at] = rest
    for part in t.view(-1).split(1 << 30):
        assert bool((part == rest).all())


def test_norm_of_the_most_rows():
    at = torch.tensor(ROWS, device="cuda")
    x, rows = sparse(at, 0)
    w = torch.randn(H, device="cuda").abs() + 0.5
    kw = dict(w_pre=w, w_post=w, alpha=0.9, beta=0.7)
    x_out, y, stats = tp.block_norm(x, [x], want_stats=True, **kw)
    del x
    want_x, want_y, want_s = tp.block_norm(rows, [rows], want_stats=True, **kw)
    same(y, at, want_y)
    del y
    nothing = tp.block_norm(torch.zeros(1, H, device="cuda", dtype=BF), [torch.zeros(1, H, device="cuda", dtype=BF)],
                            want_stats=True, **kw)[2]
    for i in range(2):
        assert torch.equal(stats[i][at], want_s[i])
        for part in stats[i].split(1 << 30):
            assert int((part != nothing[i, 0]).sum()) <= len(ROWS)
    # backward: every operand is the residual stream, so that the rest of the memory holds the results
    dx, db, dw_pre, dw_post, _ = tp.block_norm_backward(x_out, None, x_out, [x_out], stats, **kw)
    want = tp.block_norm_backward(want_x, None, want_x, [want_x], want_s, **kw)
    same(dx, at, want[0])
    same(db, at, want[1])
    same(x_out, at, want_x)
    # The same rows' terms added in another order: two roundings a row at most, of the sum of their sizes.
    d, (rb, rx) = want_x.double(), want_s.double()[:, :, None]
    xh, bh, u = (d * rx).abs(), (d * rb).abs(), (d * w).abs()
    v = 0.7 * rx * (u + xh * (u * xh).mean(1, keepdim=True))
    for got, ref, size in ((dw_pre, want[2], d.abs() * xh), (dw_post, want[3], v * bh)):
        assert ((got - ref).abs().double() <= 2 * len(ROWS) * 2.0 ** -24 * size.sum(0)).all()


def test_stash_of_the_most_rows():
    at = torch.tensor(ROWS, device="cuda")
    u, rows = sparse(at, 3)
    rows[::7] *= 300                        # blocks of different factors
    u[at] = rows
    _, (codes,), (scales,) = tp.stash_pack([u], gelu=False)
    du, h = (t[0] for t in tp.stash_backward([codes], [scales], [u]))
    # the blocks of 32 rows that hold values, by themselves
    bands = torch.unique(at // 32)
    take = (bands[:, None] * 32 + torch.arange(32, device="cuda")).view(-1)
    take = take[take < M]
    _, (want,), (byte,) = tp.stash_pack([u[take]], gelu=False)
    want_du, want_h = (t[0] for t in tp.stash_backward([want], [byte], [u[take]]))
    del u
    assert torch.equal(scales[bands], byte)
    scales[bands] = 10
    assert bool((scales == 10).all())       # nothing but zeros: the least factor
    same(du, take, want_du)
    same(h, take, want_h)
    same(codes.view(torch.uint8), take, want.view(torch.uint8))
