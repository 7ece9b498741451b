"""The tensors that the MLP block's calls return are tensors of their own: each
with its own version, none a view, and large ones with their own memory."""
import pytest
import torch

from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def pack(M, F, p=3):
    return tp.stash_pack([torch.randn(M, F, device="cuda").to(BF) for _ in range(p)])


def outputs(M, F, p=3):
    """Every call's lists of shards."""
    h, codes, scales = pack(M, F, p)
    du, act = tp.stash_backward(codes, scales, h)
    dw = tp.stash_weight_grad(codes, scales, h)
    return {"h": h, "codes": codes, "scales": scales, "du": du, "act": act, "dw": dw}


@pytest.mark.parametrize("M,F", [(5, 64), (1024, 1024)])
def test_shards_change_by_themselves(M, F):
    for name, ts in outputs(M, F).items():
        for t in ts:
            assert t._base is None and t._version == 0, name
            assert t.is_leaf and not t.requires_grad
        before = [t.clone() for t in ts]
        ts[0].zero_()
        assert ts[0]._version == 1 and [t._version for t in ts[1:]] == [0, 0], name
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ts[1:], before[1:]))


def test_a_shard_saved_for_a_gradient_outlives_changes_to_the_others():
    (h0, h1, _), *_ = pack(5, 64)
    w = torch.ones(5, 64, device="cuda", dtype=BF, requires_grad=True)
    loss = (h0 * w).sum()
    h1.zero_()
    loss.backward()
    assert torch.equal(w.grad, h0)


def test_a_large_shard_holds_its_own_memory_alone():
    large = 0
    for name, ts in outputs(2048, 2048).items():
        size = ts[1].numel() * ts[1].element_size()
        if size >= 1 << 20:
            large += 1
            held = ts[1].untyped_storage().nbytes()
            assert held == size, name
    assert large == 5                               # all but the scales
    h, codes, scales = pack(2048, 2048)
    keep, held = h[1], torch.cuda.memory_allocated()
    del h
    assert held - torch.cuda.memory_allocated() == 2 * keep.numel() * 2
