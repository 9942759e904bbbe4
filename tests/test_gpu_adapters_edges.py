"""The product with adapters in tiles of two blocks of 32 tokens whose last block does not exist."""
import numpy as np
import pytest

from test_gpu_adapters import _call, _case, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    import torch

    assert torch.cuda.is_available()
    import dual_scale_w4a4_amd

    dual_scale_w4a4_amd.lib()
    return dual_scale_w4a4_amd


# tokens, K, out, adapters, rank: odd numbers of blocks of 32 tokens, 513 .. 1024 blocks of results
SHAPES = [(65, 512, 6001, 3, 16), (96, 1024, 6000, 5, 24), (160, 512, 4096, 40, 40), (289, 512, 3001, 4, 8),
          (515, 2560, 1733, 5, 24), (545, 512, 1730, 2, 256), (1000, 512, 515, 9, 72)]


@pytest.mark.parametrize("tokens,K,out,n,rank", SHAPES)
@pytest.mark.parametrize("act_fmt,dtype", [("mxfp4", "f32"), ("mxfp4", "bf16"), ("mxfp8", "bf16")])
def test_an_odd_number_of_token_blocks(dq, tokens, K, out, n, rank, act_fmt, dtype):
    blocks = -(-tokens // 32)
    assert 512 < blocks * -(-out // 32) <= 1024
    _check(dq, _case(tokens, K, out, n, rank, act_fmt, packed=tokens % 2 == 0), dtype, residual=True)


@pytest.mark.parametrize("tokens,K,out,n,rank", SHAPES[:5])
def test_the_workspace_ends_where_its_size_says(dq, tokens, K, out, n, rank):
    # nothing behind it is written, and what lies there (NaNs) reaches no result
    import torch

    c = _case(tokens, K, out, n, rank)
    want = _call(dq, c, out_dtype="f32")
    need = dq.adapter_workspace_bytes(tokens, K, rank)
    space = torch.full((need + 65536,), 255, dtype=torch.uint8, device="cuda")
    got = _call(dq, c, out_dtype="f32", workspace=space[:need])
    assert torch.equal(got, want) and torch.all(space[need:] == 255)
    assert np.isfinite(want.cpu().numpy()).all()
