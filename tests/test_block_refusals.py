"""What is no matrix, or no tensor, is refused by name before the library is
called: host tensors suffice, since dimensions are looked at first."""
import pytest
import torch

from tensor_gemm_reduction_amd import tpfuse as tp

BF, U8, E4 = torch.bfloat16, torch.uint8, torch.float8_e4m3fn


def host(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


X, W = host(4, 64), host(64)
CODES, SCALES = host(4, 64, dtype=E4), host(1, 2, dtype=U8)
QCODES, QSCALES = host(8, 32, dtype=U8), host(8, 1)
VECTOR, SCALAR, CUBE = host(64), host(), host(2, 4, 64)


@pytest.mark.parametrize("bad,what", [(VECTOR, "has 1 dimensions"), (SCALAR, "has 0 dimensions"), (CUBE, "has 3 dimensions"),
                                      (None, "is not a tensor"), ([[0.0] * 64] * 4, "is not a tensor")])
@pytest.mark.parametrize("name,call", [
    ("x", lambda b: tp.block_norm(b, [X], W, W)),
    ("x", lambda b: tp.block_norm_backward(X, None, b, [X], host(2, 4, dtype=torch.float32), W, W)),
    (r"u\[0\]", lambda b: tp.stash_pack([b])),
    (r"codes\[0\]", lambda b: tp.stash_backward([b], [SCALES], [X])),
    (r"codes\[0\]", lambda b: tp.stash_weight_grad([b], [SCALES], [X])),
    (r"dY\[0\]", lambda b: tp.stash_weight_grad([CODES], [SCALES], [b])),
    (r"X\[0\]", lambda b: tp.qweight_matmul([b], [QCODES], [QSCALES], group=64)),
    (r"codes\[0\]", lambda b: tp.qweight_matmul([X], [b], [QSCALES], group=64)),
])
def test_matrices_are_asked_for_by_name(name, call, bad, what):
    with pytest.raises(ValueError, match=name + " " + what):
        call(bad)


@pytest.mark.parametrize("name,call", [
    ("blocks", lambda: tp.block_norm(X, [None], W, W)),
    ("w_pre", lambda: tp.block_norm(X, [X], None, W)),
    ("w_post", lambda: tp.block_norm(X, [X], W, 1.0)),
    ("gate", lambda: tp.block_norm(X, [X], W, W, gate=0.5)),
    ("dy", lambda: tp.block_norm_backward(None, None, X, [X], host(2, 4, dtype=torch.float32), W, W)),
])
def test_other_objects_are_no_operands_of_the_norm(name, call):
    with pytest.raises(ValueError, match="not a tensor|not on a GPU"):
        call()
