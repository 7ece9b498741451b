"""Outputs of the MLP block's calls come through torch's dispatcher where
something watches it, or wants new memory filled."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Log(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if isinstance(out, torch.Tensor):
            self.made.append(out.untyped_storage().data_ptr())
        return out


def test_dispatch_modes_see_the_outputs():
    x, w = torch.randn(4, 64, device="cuda").to(BF), torch.ones(64, device="cuda")
    with Log() as log:
        x_out, y, st = tp.block_norm(x, [x], w, w, want_stats=True)
        h, codes, scales = tp.stash_pack([x, x])
        yq = tp.qweight_matmul([x], [torch.zeros(8, 32, device="cuda", dtype=torch.uint8)],
                               [torch.zeros(8, 1, device="cuda", dtype=BF)], group=64)
    for t in (x_out, y, st, yq, *h, *codes, *scales):
        assert t.untyped_storage().data_ptr() in log.made


def test_uninitialized_memory_is_filled_where_asked_for():
    """torch fills new tensors in deterministic mode; outputs are whole all the same."""
    x, w = torch.randn(4, 64, device="cuda").to(BF), torch.ones(64, device="cuda")
    want = tp.block_norm(x, [x], w, w)
    torch.use_deterministic_algorithms(True)
    try:
        got = tp.block_norm(x, [x], w, w)
        filled, = tp._empty(x.device, torch.float32, (1000,))
        assert filled.isnan().all()
    finally:
        torch.use_deterministic_algorithms(False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
