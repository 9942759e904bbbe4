"""The block norm where its sums, its status word and its workspace could go wrong: squares next to
fp32's smallest, rows that hold both kinds of error, workspaces that are no dense array."""
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


@pytest.mark.parametrize("cols", [544, 2080, 16416])
@pytest.mark.parametrize("post_norm", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_overflow_beside_a_value_that_is_not_finite_is_not_reported(dq, cols, post_norm, dtype):
    """Status bit 2 is for rows whose inputs are finite: elsewhere in the row of a NaN or an infinity
    h overflows, and the other rows are clean."""
    import torch

    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    X, R = (torch.ones(5, cols, device="cuda", dtype=dt) for _ in range(2))
    gate = torch.ones(cols, device="cuda")
    for where, bad, at, over in (("X", float("nan"), 3, cols - 2), ("X", float("inf"), cols - 1, 40),
                                 ("R", float("nan"), 3, cols - 2), ("R", -float("inf"), cols - 1, 40)):
        Y, S = X.clone(), R.clone()
        S[2, over] = 3e38
        large = S.clone()
        g = gate.clone()
        g[over] = 3e38
        (Y if where == "X" else S)[2, at] = bad
        for values, want in (((Y, S), 1), ((X, large), 2), ((X, R), 0)):
            x, r = values
            codes, scales = dq.act_outputs(x, "mxfp8", 32)
            st, h = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(x)
            dq.block_norm_quantize_act_async(x, "mxfp8", 32, codes, scales, st, residual=r,
                                             residual_out=h, post_norm=post_norm,
                                             gate=None if want == 0 else g)
            # without a post norm (or with one whose output is about 1) the gate's 3e38 takes h past the
            # largest value where residual is 3e38 too
            assert int(st.item()) == want, (where, bad, at, want)


@pytest.mark.parametrize("call", ["norm_quantize_act", "block_norm_quantize_act"])
def test_a_workspace_that_is_no_dense_array_is_refused(dq, call):
    import torch

    X = torch.randn(4, 256, device="cuda")
    run = lambda ws: getattr(dq, call)(X, "mxfp8", 32, workspace=ws)  # noqa: E731
    for ws in (torch.zeros(1024, dtype=torch.uint8, device="cuda")[::4],
               torch.zeros(512, 2, dtype=torch.uint8, device="cuda").t(),
               torch.zeros(512, dtype=torch.uint8, device="cuda")[:1].expand(256)):
        with pytest.raises(ValueError, match="workspace"):
            run(ws)
    run(torch.zeros(256, dtype=torch.uint8, device="cuda"))
