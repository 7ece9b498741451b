"""The result types of the 8-bit products with sums in fp32.  No GPU: NULL handles,
pointers that are never followed."""
import pytest

from tensor_gemm_reduction_amd import tpfuse as tp
from test_expert_checks import INVALID, egrad, emm, grad, mm


@pytest.mark.parametrize("call,name", [(mm, "yt"), (emm, "yt"), (grad, "dt"), (egrad, "dt")])
@pytest.mark.parametrize("dtype,good", [(0, True), (1, True), (tp.SUMS_F32, True), (tp.SUMS_F32 + 1, True),
                                        (tp.SUMS_F32 + 2, False), (2 * tp.SUMS_F32, False), (-1, False)])
def test_result_types(call, name, dtype, good):
    assert call(**{name: dtype}) == INVALID
    said = tp.load().tpf_last_error().decode()
    assert ("handle" if good else "unknown output dtype") in said
