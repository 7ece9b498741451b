"""4-bit products of rows that hold infinities, NaN or values near the largest
finite one: every element is the sum of its own products, as in float64."""
import pytest
import torch

import block_oracle as O
from test_gpu_block import BF, F32, D, frame, qweight_case
from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu

CASES = [  # p, M, K, N, group, zeros, gelu
    (1, 1, 128, 16, 128, True, False),
    (2, 5, 160, 70, 32, True, False),
    (3, 16, 192, 4100, 64, False, False),       # 32 columns a workgroup
    (2, 20, 320, 130, 64, True, True),          # the kernel for more rows
    (2, 70, 1024, 131, 128, True, False),       # a cut contraction
    (1, 40, 2048, 100, 32, False, True),
]


def special_rows(x):
    """Rows 0, 4, 8, .. hold: +inf; -inf; both; NaN; values whose products with codes pass fp32's range."""
    inf, big, kinds = float("inf"), 2.0 ** 126, {}
    M, K = x[0].shape
    for i, m in enumerate(range(0, M, 4)):
        kinds[m] = i % 5
        if i % 5 == 0:
            x[0][m, 3] = inf
        elif i % 5 == 1:
            x[-1][m, K - 1] = -inf
        elif i % 5 == 2:
            x[0][m, 1], x[-1][m, K - 2] = inf, -inf
        elif i % 5 == 3:
            x[-1][m, 7] = float("nan")
        else:
            x[0][m, 2], x[-1][m, 5] = big, -big
    return kinds


@pytest.mark.parametrize("p,M,K,N,group,zeros,gelu", CASES)
@pytest.mark.parametrize("out", [F32, BF])
def test_each_element_is_its_own_sum(p, M, K, N, group, zeros, gelu, out):
    c = qweight_case(p, M, K, N, group, zeros, seed=11)
    kinds = special_rows(c["x"])
    y = tp.qweight_matmul(frame(c["x"]), frame(c["codes"]), frame(c["scales"]), frame(c["zeros"]) if zeros else None,
                          group=group, gelu=gelu, out_dtype=out).cpu().to(D)
    want, size = torch.zeros(M, N, dtype=D), torch.zeros(M, N, dtype=D)
    for k in range(p):
        w, wa = O.dequantize(c["codes"][k], c["scales"][k], c["zeros"][k] if zeros else None, group)
        for m in range(M):              # element by element: a matrix product may order infinities otherwise
            want[m] += (c["x"][k][m].to(D) * w).sum(1)
            size[m] += (c["x"][k][m].to(D).abs() * wa).sum(1)
    bound = (p * K + 16) * O.STEP * size            # at most one rounding a product and one a sum
    if gelu:
        bound = 1.13 * bound + 2.0 ** -20 * want.abs()
        want = want * O.cdf(want)
    if out is BF:
        bound = bound + O.half_step(BF) * want.abs()
    assert torch.equal(y.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(y[inf], want[inf])
    fin = want.isfinite()
    assert ((y - want).abs()[fin] <= bound[fin]).all()
    if M > 16:
        assert set(kinds.values()) == set(range(5))
        assert fin[16].all()            # the large values' own row
