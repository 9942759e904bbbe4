"""MLP operators on the GPU at the edges of what their documentation allows."""
import math

import numpy as np
import pytest

import mlp_ref as ref

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


# The definition 0.5 z (1 + erf(z / sqrt 2)) is 0.5 z erfc(-z / sqrt 2). Its argument in fp32 is off
# by at most 2^-23 of itself (a rounded constant and a product), which moves erfc(u) by the
# relative amount u erfc'(u) / erfc(u) < 2 u^2 + 1 = z^2 + 1 times that; the function itself is
# allowed 16 units of 2^-23 (what OpenCL asks of erfc) and the product 2^-24. Results below
# fp32's normal range count |z| 2^-126.
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _gelu(z):
    y = 0.5 * z * _erfc(-z / math.sqrt(2.0))
    return y, np.abs(y) * (2.0 ** -19 + (z * z + 1) * 2.0 ** -23 + 2.0 ** -24) + np.abs(z) * 2.0 ** -126


def _ones(dq, rows, K):
    """K ones per row as MXFP4 codes and scales, on the GPU."""
    import torch

    return (torch.full((rows, K // 2), 0x22, dtype=torch.uint8, device="cuda"),
            torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_gelu_keeps_its_precision_for_negative_values(dq, tokens):
    import torch

    out, K = 8192, 512
    print(f"[epilogue] gelu tokens={tokens}", flush=True)
    z = np.random.default_rng(5).uniform(-12.8, 12.8, out).astype(np.float32)
    z[:12] = [0.0, -1e-30, 1e-30, -4.5, -5.6, -5.7, -8.0, -12.8, 12.8, -20.0, -1e30, 1e30]
    pk = dq.gemm_pack_weights(*_ones(dq, out, K))
    y = dq.gemm_mx_epilogue(*_ones(dq, tokens, K), pk, a=torch.zeros(out, device="cuda"),
                            bias=torch.from_numpy(z).cuda(), activation="gelu", out_dtype="f32")
    got = y.double().cpu().numpy()
    want, dy = _gelu(z.astype(np.float64))
    bad = np.argwhere(~(np.abs(got - want) <= dy))
    assert bad.size == 0, (len(bad), [(z[c], got[t, c], want[c]) for t, c in bad[:6]])
    nz = np.abs(want) > 2.0 ** -120
    print("largest relative error", (np.abs(got - want)[:, nz] / np.abs(want[nz])).max())


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("tokens", [1, 300, 700])  # each kernel: split, tiles of 64 and of 128
def test_gated_gelu_quantizes_groups_of_negative_gates(dq, fmt, tokens):
    # the gate of group j lies in [-8 + j / 32, -8 + (j + 1) / 32]; sums of 512 ones are exact
    import torch

    K, inner = 512, 4096
    print(f"[gated] gelu tokens={tokens} {fmt}", flush=True)
    rng = np.random.default_rng(6)
    z = (-8.0 + (np.arange(inner) // 32 + rng.random(inner)) / 32).astype(np.float32)
    u = rng.uniform(0.5, 2.0, inner).astype(np.float32)
    pk = dq.gemm_pack_weights(*_ones(dq, inner, K))
    dev = lambda v: torch.from_numpy(v / np.float32(K)).cuda()  # noqa: E731
    q = dq.gated_mx_quantized(*_ones(dq, tokens, K), pk, pk, fmt, a_gate=dev(z), a_up=dev(u),
                              activation="gelu")
    g, dg = _gelu(z.astype(np.float64))
    want, dx = g * u, dg * u + np.abs(g * u) * ref.U24
    codes, scales = q["codes"].cpu().numpy(), q["scales"].cpu().numpy()
    assert np.all(codes == codes[0]) and np.all(scales == scales[0])
    ref.check_quantized(codes[:1], scales[:1], want[None], dx[None], fmt)


@pytest.mark.parametrize("tokens", [1, 60, 300, 700])  # each kernel of the selection
@pytest.mark.parametrize("act_fmt", ["mxfp4", "mxfp8"])
def test_products_repeat_themselves_bit_for_bit(dq, tokens, act_fmt):
    # eager calls among others, on other outputs, and replays of a graph
    import torch

    K, channels = 2560, 4096
    print(f"[repeat] tokens={tokens} {act_fmt}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, K, device="cuda", generator=g)
    q = dq.norm_quantize_act(x, act_fmt, 32)
    w = dq.quantize_act(torch.randn(channels, K, device="cuda", generator=g), "mxfp4", 32)
    pk = dq.gemm_pack_weights(w["codes"], w["scales"])

    def run():
        kw = dict(act_fmt=act_fmt)
        y = dq.gemm_mx_epilogue(q["codes"], q["scales"], pk, activation="gelu", **kw)
        m = dq.gated_mx_quantized(q["codes"], q["scales"], pk, pk, "mxfp8", **kw)
        return y, dq.gated_mx(q["codes"], q["scales"], pk, pk, **kw), m["codes"], m["scales"]

    first = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(4):
        graph.replay()
        again = run()
        torch.cuda.synchronize()
        for got in (captured, again):
            assert all(torch.equal(a, b) for a, b in zip(first, got))
