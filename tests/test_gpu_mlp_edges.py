"""MLP operators on the GPU at the edges of what their documentation allows."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    import torch

    assert torch.cuda.is_available()
    import dual_scale_w4a4_amd

    dual_scale_w4a4_amd.lib()
    return dual_scale_w4a4_amd


@pytest.mark.parametrize("cols", [1056, 4128, 8160])  # several waves, the last one not full
@pytest.mark.parametrize("tokens", [1, 5, 3000])      # 3000: several rows per workgroup
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("into", ["X", "residual"])
def test_norm_in_place_reports_no_value_that_no_row_holds(dq, cols, tokens, dtype, into):
    # h = X + R stays below the largest fp32 where h + R or h + X, which exist only if a lane
    # adds to a row that has been updated already, would not
    import torch

    print(f"[norm] in place {tokens}x{cols} {dtype} into {into}", flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(cols + tokens)
    X = torch.randn(tokens, cols, device="cuda", generator=g).to(dt)
    R = torch.randn(tokens, cols, device="cuda", generator=g).to(dt)
    X[:, :16] = 1.25e38
    R[:, :16] = 1.25e38
    want = dq.norm_quantize_act(X, "mxfp8", 32, residual=R)
    assert torch.equal(want["residual"], (X.float() + R.float()).to(dt))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = dq.act_outputs(X, "mxfp8", 32)
    h = X if into == "X" else R
    dq.norm_quantize_act_async(X, "mxfp8", 32, codes, scales, status, residual=R, residual_out=h)
    assert int(status.item()) == 0
    assert torch.equal(h, want["residual"])
    assert torch.equal(codes, want["codes"]) and torch.equal(scales, want["scales"])
