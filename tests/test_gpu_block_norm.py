"""The block norm on the GPU against its definition (layer_ref.py), bit for bit: both norms, the
gates, the scaled residual, x_out and the quantizer."""
import numpy as np
import pytest

import layer_ref
import mlp_ref as ref
from parity import host, scales_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    import torch

    assert torch.cuda.is_available()
    import dual_scale_w4a4_amd

    dual_scale_w4a4_amd.lib()
    return dual_scale_w4a4_amd


def _tensor(x, dtype="f32"):
    import torch

    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def _numpy(t):
    return t.float().cpu().numpy()


def _case(tokens, cols, dtype, seed, wdt="f32", **off):
    """Seeded inputs of every array, as float32 values of their types; off: arrays left out."""
    rng = np.random.default_rng(seed)
    level = np.exp(0.5 * rng.standard_normal(cols))
    level[rng.random(cols) < 0.02] *= 20
    c = dict(X=layer_ref.rounded((rng.standard_normal((tokens, cols)) * level).astype(np.float32), dtype),
             R=layer_ref.rounded((rng.standard_normal((tokens, cols)) * level).astype(np.float32), dtype),
             post=layer_ref.rounded((1 + 0.3 * rng.standard_normal(cols)).astype(np.float32), wdt),
             w=layer_ref.rounded((1 + 0.3 * rng.standard_normal(cols)).astype(np.float32), wdt),
             gate=np.tanh(rng.standard_normal(cols)).astype(np.float32),
             tgate=rng.random(tokens).astype(np.float32),
             b=np.ldexp(np.float32(1), rng.integers(-3, 4, cols)).astype(np.float32))
    c.update({k: None for k, v in off.items() if not v})
    return dict(c, dtype=dtype, wdt=wdt, rs=0.8125)


def _quantized(oracle, x, fmt, group, g):
    if fmt == "mxfp8":
        return ref.mxfp8(x, group)
    q = oracle.quantize_act(x, "f32", fmt, group, None, g)
    return q["codes"], q["scales"]


def _check(dq, oracle, c, fmt, group=32, g=0.0, post_norm=True, xdt=None, inplace=None, eps=1e-5,
           post_eps=1e-6, where=None):
    import torch

    tokens, cols = c["X"].shape
    print(f"[block norm] {tokens}x{cols} {c['dtype']} {fmt} G={group} post={post_norm} xdt={xdt} "
          f"inplace={inplace} off={[k for k, v in c.items() if v is None]}", flush=True)
    X, R = _tensor(c["X"], c["dtype"]), _tensor(c["R"], c["dtype"])
    x_out = None if xdt is None else torch.empty(
        X.shape, dtype=torch.bfloat16 if xdt == "bf16" else torch.float32, device="cuda")
    out = {"R": R, "X": X, None: None}[inplace]
    post = c["post"] if post_norm else None
    got = dq.block_norm_quantize_act(
        X, fmt, group, residual=R, residual_out=out, post_norm=post_norm,
        post_weight=_tensor(post, c["wdt"]), post_eps=post_eps, gate=_tensor(c["gate"]),
        token_gate=_tensor(c["tgate"]), residual_scale=c["rs"], weight=_tensor(c["w"], c["wdt"]),
        eps=eps, x_out=x_out, b=_tensor(c["b"]), g=g)
    torch.cuda.synchronize()
    h, n, x = layer_ref.block_norm(c["X"], c["R"], post, c["gate"], c["tgate"], c["rs"], c["w"],
                                   c["b"], c["dtype"], post_norm, post_eps, eps)
    codes, scales = _quantized(oracle, x, fmt, group, g)
    if out is not None:
        assert got["residual"] is out
    assert np.array_equal(_numpy(got["residual"]), h)
    if xdt is not None:
        assert got["x"] is x_out and np.array_equal(_numpy(x_out), layer_ref.rounded(n, xdt))
    bad = np.argwhere(host(got["codes"]) != codes)
    assert bad.size == 0, (len(bad), bad[:4])
    assert np.array_equal(scales_np(got["scales"], fmt), scales)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "mxint4", "nvfp4", "int4_bf16"])
@pytest.mark.parametrize("group", [16, 32, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_format(dq, oracle_lib, fmt, group, dtype):
    c = _case(19, 1088, dtype, group, wdt=dtype)
    _check(dq, oracle_lib, c, fmt, group, g=0.004 if fmt == "nvfp4" else 0.0, xdt=dtype)


@pytest.mark.parametrize("tokens,cols", [(1, 16), (1, 64), (3, 96), (5, 1024), (2, 1056), (7, 4096),
                                         (3, 4112), (2, 8192), (2, 8208), (3, 14336), (2, 16384),
                                         (2, 16400), (1, 40960), (1100, 4096), (2050, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shapes(dq, oracle_lib, tokens, cols, dtype):
    group = 32 if cols % 32 == 0 else 16
    c = _case(tokens, cols, dtype, cols + tokens)
    for k, inplace in enumerate((None, "R", "X") if tokens < 100 else ("R",)):
        _check(dq, oracle_lib, c, ("mxfp8", "mxfp4", "mxfp8")[k], group, post_norm=k != 1,
               xdt=(None, "bf16", "f32")[k], inplace=inplace)


@pytest.mark.parametrize("mask", range(32))
def test_each_array_may_be_left_out(dq, oracle_lib, mask):
    for dtype, cols in (("bf16", 544), ("f32", 16416)):
        c = _case(3, cols, dtype, mask, wdt=("f32", "bf16")[mask % 2], R=mask & 1, post=mask & 2,
                  gate=mask & 4, tgate=mask & 8, w=mask & 16, b=mask & 1)
        _check(dq, oracle_lib, c, "mxfp8", xdt="bf16" if mask & 2 else "f32")
        if mask % 5 == 0:
            _check(dq, oracle_lib, c, "mxfp4", post_norm=False)


def test_without_post_norm_and_gates_it_is_the_single_norm(dq):
    import torch

    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(33, 2080, device="cuda", generator=g).to(torch.bfloat16)
    R = torch.randn(33, 2080, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.rand(2080, device="cuda", generator=g) + 0.5
    a = dq.norm_quantize_act(X, "mxfp4", 32, weight=w, residual=R, eps=1e-6)
    b = dq.block_norm_quantize_act(X, "mxfp4", 32, residual=R, post_norm=False, weight=w, eps=1e-6)
    for k in ("codes", "scales", "residual"):
        assert torch.equal(a[k], b[k])


def test_rows_of_zeros_and_extreme_values(dq, oracle_lib):
    cols = 1024
    rng = np.random.default_rng(5)
    X, R = np.zeros((6, cols), np.float32), np.zeros((6, cols), np.float32)
    X[1] = 2.0 ** -149
    X[2] = 1e38 * np.sign(rng.standard_normal(cols))
    R[3] = rng.standard_normal(cols)
    X[4, 100:130] = rng.standard_normal(30)
    X[5, ::3], R[5] = -1e-42, 1e-30
    c = dict(_case(6, cols, "f32", 1), X=X, R=R)
    for fmt in ("mxfp8", "mxfp4", "mxint4"):
        for post_norm in (True, False):
            _check(dq, oracle_lib, c, fmt, post_norm=post_norm, xdt="f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [1024, 16416])
def test_every_magnitude(dq, oracle_lib, dtype, cols):
    # rows, and parts of rows, of every magnitude, around those where squares leave fp32's range
    powers = [-140, -126, -100, -76, -75, -64, -63, -52, -51, -50, -49, -20, 0, 30, 61, 62, 63, 64, 100, 120]
    rng = np.random.default_rng(cols)
    X = rng.standard_normal((len(powers), cols)) * np.exp2(np.array(powers, float))[:, None]
    X[3, ::7] *= 2.0 ** 40
    X[12, 100:300] *= 2.0 ** -90
    X[14, 5] *= 2.0 ** 50
    R = rng.standard_normal((len(powers), cols)) * np.exp2(np.array(powers[::-1], float))[:, None]
    R[5:9] = 0
    c = dict(_case(len(powers), cols, dtype, 3), X=layer_ref.rounded(X.astype(np.float32), dtype),
             R=layer_ref.rounded(R.astype(np.float32), dtype))
    for post_norm in (True, False):
        for eps in (1e-5, 1e-75):  # 1 / sqrt(eps) has to fit fp32, where the definition rounds it to
            _check(dq, oracle_lib, c, "mxfp8", post_norm=post_norm, xdt="f32", eps=eps, post_eps=eps)


def test_many_rows(dq, oracle_lib):
    # a wrong last bit of either root shows in some row
    for dtype, cols in (("bf16", 512), ("f32", 352)):
        _check(dq, oracle_lib, _case(20000, cols, dtype, 9), "mxfp8", xdt="f32")


@pytest.mark.parametrize("cols", [544, 2080, 16416])
@pytest.mark.parametrize("post_norm", [True, False])
def test_errors_are_reported_and_other_rows_are_right(dq, cols, post_norm):
    import torch

    clean = _case(9, cols, "f32", 7)

    def run(X, R, **kw):
        codes, scales = dq.act_outputs(X, "mxfp8", 32)
        st, h = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(X)
        dq.block_norm_quantize_act_async(X, "mxfp8", 32, codes, scales, st, residual=R,
                                         residual_out=h, post_norm=post_norm, **kw)
        return codes, scales, h, int(st.item())

    X, R = _tensor(clean["X"]), _tensor(clean["R"])
    want = run(X, R)
    assert want[3] == 0
    others = [r for r in range(9) if r != 4]
    for which in "XR":
        for bad in (float("nan"), float("inf"), -float("inf")):
            for at in (0, cols // 2 + 1, cols - 1):
                Y, S = X.clone(), R.clone()
                (Y if which == "X" else S)[4, at] = bad
                got = run(Y, S)
                assert got[3] == 1, (which, bad, at, got[3])
                for a, b in zip(got[:3], want[:3]):
                    assert torch.equal(a[others], b[others])
    big = R.clone()
    big[4] = 3e38
    got = run(X if post_norm else torch.where(big > 1e38, big, X), big, gate=torch.full(
        (cols,), 3e38, device="cuda"))  # h overflows
    assert got[3] == 2
    got = run(X, R, weight=torch.full((cols,), 3e38, device="cuda"))  # n overflows
    assert got[3] == 2
    b = torch.full((cols,), 3e38, device="cuda")
    assert run(X, R, b=b)[3] == 2                                     # x overflows
    with pytest.raises(dq.DQError, match="RANGE"):
        dq.block_norm_quantize_act(X, "mxfp8", 32, residual=R, post_norm=post_norm, b=b)
    Y = X.clone()
    Y[0, 0] = float("nan")
    with pytest.raises(dq.DQError, match="NONFINITE"):
        dq.block_norm_quantize_act(Y, "mxfp8", 32, residual=R, post_norm=post_norm)
    # a value of n that only its rounding to bf16 takes past the largest: reported where stored
    one = torch.ones(1, 32, device="cuda")
    w = torch.full((32,), 3.4e38, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = dq.act_outputs(one, "mxfp8", 32)
    for x_out, bits in ((None, 0), (torch.empty(1, 32, dtype=torch.bfloat16, device="cuda"), 2)):
        dq.block_norm_quantize_act_async(one, "mxfp8", 32, codes, scales, st, post_norm=False,
                                         residual_out=torch.empty_like(one), weight=w, x_out=x_out)
        assert int(st.item()) == bits


def test_streams_and_workspace(dq):
    import torch

    c = _case(40, 4096, "bf16", 3)
    X, R = _tensor(c["X"], "bf16"), _tensor(c["R"], "bf16")
    want = dq.block_norm_quantize_act(X, "mxfp4", 32, residual=R)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    got = dq.block_norm_quantize_act(X, "mxfp4", 32, residual=R, workspace=ws, stream=s)
    for k in want:
        assert torch.equal(got[k], want[k])


def test_graph_replays(dq):
    import torch

    c = _case(5, 4096, "bf16", 4)
    X, R = _tensor(c["X"], "bf16"), _tensor(c["R"], "bf16")
    codes, scales = dq.act_outputs(X, "mxfp8", 32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, x = torch.empty_like(X), torch.empty_like(X)
    call = lambda: dq.block_norm_quantize_act_async(X, "mxfp8", 32, codes, scales, st, residual=R,  # noqa: E731
                                                    residual_out=h, x_out=x, residual_scale=0.5)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        X.copy_(torch.randn(5, 4096, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (codes, scales, h, x)]
        for t in (codes, scales, h, x):
            t.zero_()
        call()
        torch.cuda.synchronize()
        for a, b in zip(got, (codes, scales, h, x)):
            assert torch.equal(a, b), k
    assert int(st.item()) == 0
