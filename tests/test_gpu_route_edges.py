"""The router's kernels with bounds where a bound could be wrong or worth nothing: rows of zeros, as a
padded batch has them, and values below fp32's normal range."""
import numpy as np
import pytest

import layer_ref
import mlp_ref as ref
from test_gpu_route import _check_result, _tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    import torch

    assert torch.cuda.is_available()
    import dual_scale_w4a4_amd

    dual_scale_w4a4_amd.lib()
    return dual_scale_w4a4_amd


# above 2^16 logits and 2^28 products: tokens, channels, experts, top k
SHAPES = [(1100, 4096, 64, 8), (900, 2600, 130, 6), (1500, 4096, 128, 8), (300, 1032, 1000, 32)]


@pytest.mark.parametrize("tokens,cols,experts,top_k", SHAPES)
@pytest.mark.parametrize("score,bias", [("sigmoid", True), ("sigmoid", False), ("softmax", False)])
def test_rows_of_zeros(dq, tokens, cols, experts, top_k, score, bias):
    # tokens of a padded batch, experts whose rows are zeros, and negative zeros among both
    rng = np.random.default_rng(tokens)
    X = ref.bf16(rng.standard_normal((tokens, cols)).astype(np.float32))
    W = ref.bf16((rng.standard_normal((experts, cols)) * 1.5 / np.sqrt(cols)).astype(np.float32))
    X[tokens // 2:] *= 0.0
    X[5, 17:] = 0.0
    W[[1, experts - 1]] *= 0.0
    b = (0.1 * rng.standard_normal(experts)).astype(np.float32) if bias else None
    if bias:
        b[7] = b[3]
    got = dq.moe_route(_tensor(X, "bf16"), _tensor(W, "bf16"), top_k, score=score, bias=_tensor(b))
    _check_result(got, X, W, top_k, score, b)
    if not bias:
        assert np.array_equal(got[0][-1].cpu().numpy(), np.arange(top_k))


@pytest.mark.parametrize("tokens,cols,experts,top_k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("small", ["X", "W"])
def test_values_below_fp32_normal_range_count(dq, tokens, cols, experts, top_k, score, small):
    # subnormal values of one operand times large ones of the other: products next to 1
    rng = np.random.default_rng(experts)
    tiny = np.ldexp(rng.integers(-100, 101, (tokens, cols) if small == "X" else (experts, cols)).astype(
        np.float32), -133)
    large = rng.standard_normal((experts, cols) if small == "X" else (tokens, cols))
    large = ref.bf16((large * 2.0 ** 126 / np.sqrt(cols)).astype(np.float32))
    X, W = (tiny, large) if small == "X" else (large, tiny)
    X = X.copy()
    X[::3] = ref.bf16((rng.standard_normal(X[::3].shape) * (2.0 ** -122 if small == "X" else 2.0 ** 120)
                       ).astype(np.float32))
    got = dq.moe_route(_tensor(X, "bf16"), _tensor(W, "bf16"), top_k, score=score)
    assert np.abs(layer_ref.logits(X, W)).max() > 0.1
    _check_result(got, X, W, top_k, score)


def test_products_below_fp32_range_are_within_the_bound(dq):
    # every product underflows fp32; the fp64 sums order the experts
    tokens, cols, experts = 700, 4096, 96
    rng = np.random.default_rng(2)
    X = ref.bf16((rng.standard_normal((tokens, cols)) * 2.0 ** -75).astype(np.float32))
    W = ref.bf16((rng.standard_normal((experts, cols)) * 2.0 ** -75).astype(np.float32))
    X[0, 0], W[3, 0] = 2.0 ** -70, 2.0 ** -60
    for score in ("softmax", "sigmoid"):
        got = dq.moe_route(_tensor(X, "bf16"), _tensor(W, "bf16"), 5, score=score)
        _check_result(got, X, W, 5, score)


@pytest.mark.parametrize("tokens,cols,experts,top_k", [(4096, 4096, 128, 8), (1024, 7168, 256, 8)])
def test_a_padded_batch_takes_no_longer(dq, tokens, cols, experts, top_k):
    # every expert of a token of zeros is in question; summing them all again took 3 to 9 times as long
    import torch

    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(tokens, cols, device="cuda", generator=g).to(torch.bfloat16)
    W = (torch.randn(experts, cols, device="cuda", generator=g) * 1.5 / cols ** 0.5).to(torch.bfloat16)
    out = dict(ids=torch.empty(tokens, top_k, dtype=torch.int32, device="cuda"),
               weights=torch.empty(tokens, top_k, device="cuda"),
               workspace=torch.empty(dq.moe_route_workspace_bytes(tokens, experts), dtype=torch.uint8,
                                     device="cuda"))

    def least_ms(x):
        times = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(20):
                dq.moe_route(x, W, top_k, score="sigmoid", **out)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    full = least_ms(X)
    for part in (0.1, 0.5, 1.0):
        padded = X.clone()
        padded[tokens - int(part * tokens):] = 0
        assert least_ms(padded) < 2 * full, part
