"""The binding's native argument checks, on the CPU: they find no operands in
what is not a contiguous GPU tensor of the asked-for kind, and name misuse."""
import pytest
import torch

from tensor_gemm_reduction_amd import tpfuse as tp


def native():
    tp.load()
    return tp._args


def test_host_tensors_and_other_objects_are_no_operands():
    n, t = native(), torch.zeros(3, 4)
    assert n.operands(0, (t,), torch.float32, (3, 4)) is None
    for what in ((1,), (None,), ("x",), ([t],)):
        assert n.operands(0, what, torch.float32, (3, 4)) is None
    assert n.operands(0, 7, torch.float32, (3, 4)) is None              # not a sequence
    assert n.operands(0, (t,), "float32", (3, 4)) is None
    assert n.operands(0, (t,), torch.float32, [3, 4]) is None
    assert n.operands(0, (t,), torch.float32, ("a", 4)) is None
    assert n.operands(0, (t,), torch.float32, (2 ** 70, 4)) is None
    assert n.operands(0, (t.to_sparse(),), torch.float32, (3, 4)) is None
    assert n.operands(0, (t.to("meta"),), torch.float32, (3, 4)) is None


def test_no_tensors_have_no_addresses():
    assert native().operands(0) == ()
    assert native().operands(0, (), torch.float32, (3, 4), [], torch.uint8, ()) == (b"", b"")


@pytest.mark.parametrize("args", [(), (0, (), torch.float32), ("0",)])
def test_operands_misuse(args):
    with pytest.raises(TypeError):
        native().operands(*args)


@pytest.mark.parametrize("args", [(), (0, torch.float32), (0, "f", (2,)), (0, torch.float32, [2]), (0, torch.float32, ("a",)),
                                  (0.5,)])
def test_empty_misuse(args):
    with pytest.raises(TypeError):
        native().empty(*args)


@pytest.mark.parametrize("args", [(0,), (0, 2, torch.float32), (0, 2, "f", (2,)), (0, 2, torch.float32, 3)])
def test_shards_misuse(args):
    with pytest.raises(TypeError):
        native().shards(*args)


def test_empty_of_nothing():
    assert native().empty(0, torch.float32, None) == (None,)
