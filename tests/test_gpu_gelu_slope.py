"""GeLU's gradient from the 8-bit activations where it is small: near the zero
of the slope Phi(u) + u phi(u) its two terms cancel, so an error of theirs that
is small beside a bf16 step of either is large beside a step of the result."""
import pytest
import torch

import block_oracle as O
from tensor_gemm_reduction_amd import tpfuse as tp

pytestmark = pytest.mark.gpu
D = torch.float64


@pytest.mark.parametrize("exponent", [124, 126, 127, 129])
def test_gelu_slope_to_single_precision(exponent):
    """Every e4m3 value times a power of two, 512 gradients for each."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(512, 1)
    codes = torch.where((codes & 127) == 127, torch.zeros_like(codes), codes)      # no NaN
    scales = torch.full((16, 8), exponent, dtype=torch.uint8)
    g = torch.Generator().manual_seed(exponent)
    dh = torch.randn(512, 256, generator=g).bfloat16()
    (du,), (h,) = tp.stash_backward([codes.cuda().view(torch.float8_e4m3fn)], [scales.cuda()], [dh.cuda()])
    u = O.unpack(codes.view(torch.float8_e4m3fn).float(), scales)
    near = u.abs() <= 4
    assert near.sum() > 1000
    d = dh.to(D)
    want, size = d * (O.cdf(u) + u * O.pdf(u)), d.abs() * (O.cdf(u) + u.abs() * O.pdf(u))
    # Roundings of fp32 in Phi: 3 in the polynomial's argument, 4 in its steps and fit, 2 products; in
    # exp(-u^2 / 2) 2, and up to 2 of its argument, which count u^2 / 2 each; in u phi 2 more, in the sum 1,
    # in the product with the gradient 1.
    steps = 16 + 2 * u * u
    bound = O.half_step(torch.bfloat16) * want.abs() + steps * O.STEP * size
    bad = (du.cpu().to(D) - want).abs() > bound
    assert not bad[near].any(), f"{int(bad[near].sum())} of {int(near.sum())} gradients out, u = " \
                                f"{sorted(set(u[bad & near].tolist()))[:8]}"
    value, vsize = u * O.cdf(u), (u * O.cdf(u)).abs()
    bad = (h.cpu().to(D) - value).abs() > (O.half_step(torch.bfloat16) + steps * O.STEP) * vsize + 2.0 ** -126
    assert not bad[near].any()
