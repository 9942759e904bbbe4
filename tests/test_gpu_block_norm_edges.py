"""The block norm where its sums could go wrong: squares next to fp32's smallest."""
from fractions import Fraction

import numpy as np
import pytest

import layer_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    import torch

    assert torch.cuda.is_available()
    import dual_scale_w4a4_amd

    dual_scale_w4a4_amd.lib()
    return dual_scale_w4a4_amd


@pytest.mark.parametrize("power", [-50, -49])
@pytest.mark.parametrize("cols", [64, 1024, 16448])
def test_squares_below_fp32_normal_range_count(dq, power, cols):
    """One value in 16 is 1.5 2^power, the others' squares are 7.39 2^-149, which fp32 rounds to a
    subnormal. eps puts the root so near to a midpoint of two fp32 numbers that the small squares
    (2^-43 of the sum and less) decide to which it rounds."""
    import torch

    big, small = 1.5 * 2.0 ** power, 1.921875 * 2.0 ** -74
    X = np.full((1, cols), small, np.float32)
    X[0, ::16] = big
    large, rest = Fraction(big) ** 2 / 16, Fraction(small) ** 2 * 15 / 16  # of the mean
    mean = large + rest
    r = np.float32(1 / np.sqrt(2 * float(mean)))  # so that eps is about the mean
    middle = (Fraction(float(r)) + Fraction(float(np.nextafter(r, np.float32(0))))) / 2
    eps = float(1 / middle ** 2 + rest / 2 - mean)
    # fl32 of the root with and without the small squares: far apart next to fp64's roundings
    v = [float(np.float32(1 / np.sqrt(float(m + Fraction(eps))))) for m in (mean, large)]
    assert v[0] != v[1]
    x_out = torch.empty(1, cols, device="cuda")
    got = dq.block_norm_quantize_act(torch.from_numpy(X).cuda().to(torch.bfloat16), "mxfp8", 32,
                                     post_norm=False, eps=eps, x_out=x_out)
    torch.cuda.synchronize()
    h, n, _ = layer_ref.block_norm(X, None, None, None, None, 1.0, None, None, "bf16", False, 1.0, eps)
    assert np.array_equal(got["residual"].float().cpu().numpy(), h)
    assert n[0, 0] == np.float32(big) * np.float32(v[0])
    assert np.array_equal(x_out.cpu().numpy(), n)
