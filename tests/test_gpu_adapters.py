"""The product with low-rank adapters on the GPU against a plain float64 implementation
(layer_ref.adapters), within the bound that its arithmetic gives, and exactly where every sum is."""
import numpy as np
import pytest

import layer_ref
import mlp_ref as ref
import workloads
from parity import to_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    import torch

    assert torch.cuda.is_available()
    import dual_scale_w4a4_amd

    dual_scale_w4a4_amd.lib()
    return dual_scale_w4a4_amd


def _dev(a):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bf16(x):
    """float32 values that are bf16, on the device"""
    x = np.ascontiguousarray(x, np.float32)
    return to_device((x.view(np.uint32) >> 16).astype(np.uint16), "bf16")


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _case(tokens, K, out, n, rank, act_fmt="mxfp4", seed=0, packed=False, none=0.15):
    rng = np.random.default_rng(seed + 11 * tokens + rank)
    xc, xs = (workloads.mx_operands(tokens, K, seed=seed + 1, lo=124, hi=130) if act_fmt == "mxfp4"
              else ref.mxfp8_operand(rng, tokens, K))
    wc, ws = workloads.mx_operands(out, K, seed=seed + 2, lo=118, hi=124)
    a = (rng.uniform(0.1, 1.5, out) / np.sqrt(K)).astype(np.float32)
    r = lambda *s: ref.bf16(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    adapter = rng.integers(0, n, tokens)
    if packed:
        adapter = np.sort(adapter)
    adapter[rng.random(tokens) < none] = -1
    return dict(xc=xc, xs=xs, wc=wc, ws=ws, a=a, act_fmt=act_fmt, X=r(tokens, K),
                A=ref.bf16(r(n, rank, K) / np.float32(np.sqrt(K))), B=r(n, out, rank),
                scale=rng.uniform(0.25, 2, n).astype(np.float32),
                adapter=adapter.astype(np.int32))


def _call(dq, c, **kw):
    return dq.gemm_mx_adapters(_dev(c["xc"]), _dev(c["xs"]), dq.gemm_pack_weights(_dev(c["wc"]), _dev(c["ws"])),
                               _bf16(c["X"]), _dev(c["adapter"]), _bf16(c["A"]), _bf16(c["B"]),
                               scale=_dev(c["scale"]), a=_dev(c["a"]), act_fmt=c["act_fmt"], **kw)


def _sampled(n, sample, seed=1):
    if n <= sample:
        return np.arange(n)
    rng = np.random.default_rng(seed)
    return np.unique(np.concatenate([rng.choice(n, sample - 4, replace=False), [0, 31, n - 2, n - 1]]))


def _check(dq, c, dtype="bf16", kind="none", bias=False, residual=False, inplace=False, sample=200):
    tokens, out = c["xc"].shape[0], c["wc"].shape[0]
    n, rank, K = c["A"].shape
    print(f"[adapters] {tokens} x {K} -> {out}, {n} of rank {rank}, {c['act_fmt']}->{dtype} {kind} "
          f"bias={bias} residual={residual}", flush=True)
    rng = np.random.default_rng(tokens)
    bv = rng.standard_normal(out).astype(np.float32) if bias else None
    rh = rd = None
    if residual:
        rh = layer_ref.rounded(rng.standard_normal((tokens, out)).astype(np.float32), dtype)
        rd = _bf16(rh) if dtype == "bf16" else _dev(rh)
    y = _call(dq, c, bias=_dev(bv), activation=kind, residual=rd, out_dtype=dtype,
              y=rd if inplace else None)
    ts, cs = _sampled(tokens, sample), _sampled(out, sample)
    want, dy = layer_ref.adapters(
        c["xc"][ts], c["xs"][ts], c["act_fmt"], c["wc"][cs], c["ws"][cs],
        None if c["a"] is None else c["a"][cs], None if bv is None else bv[cs], kind,
        None if rh is None else rh[np.ix_(ts, cs)], c["X"][ts], c["adapter"][ts], c["A"],
        c["B"][:, cs], c["scale"], dtype)
    ref.check_rounded(_f64(y)[np.ix_(ts, cs)], want, dy, dtype)
    return y


# tokens, K, out, adapters, rank: every kernel of the product's selection, ranks that end inside a step
# of 16 and a block of 32, more adapters than a block of tokens, one adapter, odd channels
SHAPES = [(1, 512, 4, 1, 8), (1, 2048, 70, 3, 16), (2, 512, 1000, 40, 24), (17, 1536, 33, 17, 64),
          (32, 512, 256, 64, 16), (33, 1024, 260, 5, 40), (64, 2560, 96, 100, 8), (97, 512, 131, 2, 128),
          (130, 1024, 300, 7, 256), (300, 512, 520, 30, 32), (160, 512, 3200, 4, 48),
          (333, 1024, 4004, 9, 16), (510, 512, 6000, 3, 72), (700, 512, 9001, 12, 16),
          (1030, 512, 5555, 200, 8)]


@pytest.mark.parametrize("tokens,K,out,n,rank", SHAPES)
@pytest.mark.parametrize("act_fmt,dtype", [("mxfp4", "bf16"), ("mxfp4", "f32"), ("mxfp8", "bf16")])
def test_shapes(dq, tokens, K, out, n, rank, act_fmt, dtype):
    c = _case(tokens, K, out, n, rank, act_fmt, packed=tokens % 2 == 0)
    _check(dq, c, dtype, residual=True, inplace=tokens % 3 == 0)


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,out", [(5, 100), (290, 4100)])
def test_activations_and_optional_arrays(dq, kind, dtype, tokens, out):
    c = _case(tokens, 512, out, 4, 16)
    _check(dq, c, dtype, kind, bias=True)
    _check(dq, dict(c, a=None, scale=None), dtype, kind, bias=kind == "silu", residual=True)


@pytest.mark.parametrize("tokens,out", [(1, 64), (40, 70), (100, 300), (300, 2100), (300, 4100),
                                        (1100, 4099)])
@pytest.mark.parametrize("rank", [8, 40])
def test_exact_where_the_sums_are(dq, tokens, out, rank):
    # integers whose sums stay below 2^24: u up to 23 bits, which only its whole split carries
    n, K = 6, 512
    rng = np.random.default_rng(rank + tokens)
    c = _case(tokens, K, out, n, rank, seed=3)
    c["X"] = rng.integers(-90, 91, (tokens, K)).astype(np.float32)
    c["A"] = rng.integers(-90, 91, (n, rank, K)).astype(np.float32)
    c["B"] = np.zeros((n, out, rank), np.float32)
    np.put_along_axis(c["B"], rng.integers(0, rank, (n, out, 1)), 1.0, 2)
    c["scale"] = (2.0 ** rng.integers(-1, 2, n)).astype(np.float32)
    c["a"] = np.zeros(out, np.float32)
    y = _f64(_call(dq, c, out_dtype="f32"))
    want = np.zeros((tokens, out))
    for r in range(n):
        t = c["adapter"] == r
        want[t] = c["X"][t].astype(np.float64) @ c["A"][r].T.astype(np.float64) @ c["B"][r].T * c["scale"][r]
    assert np.abs(want).max() > 2 ** 16
    assert np.array_equal(y, want)


@pytest.mark.parametrize("tokens", [30, 300])
def test_tokens_without_an_adapter_are_the_shared_product(dq, tokens):
    import torch

    c = _case(tokens, 512, 264, 3, 16, seed=5)
    c["adapter"] = np.random.default_rng(1).choice(
        [-1, -2 ** 31, 3, 2 ** 31 - 1, 1], tokens).astype(np.int32)
    c["a"] = np.exp2(np.round(np.log2(c["a"]))).astype(np.float32)  # exact products with it
    for dtype in ("bf16", "f32"):
        y = _check(dq, c, dtype)
        plain = dq.gemm_mx_epilogue(_dev(c["xc"]), _dev(c["xs"]),
                                    dq.gemm_pack_weights(_dev(c["wc"]), _dev(c["ws"])),
                                    a=_dev(c["a"]), out_dtype=dtype)
        none = torch.from_numpy(c["adapter"] != 1).cuda()
        assert torch.equal(y[none], plain[none])
        assert not torch.equal(y[~none], plain[~none])


@pytest.mark.parametrize("tokens,out", [(20, 64), (300, 4100)])
def test_nan_and_infinities_reach_their_own_tokens_only(dq, tokens, out):
    c = _case(tokens, 512, out, 5, 24, seed=7, none=0.2)
    clean = _f64(_call(dq, c))
    for name, at, value in (("A", (2, 3, 100), np.nan), ("B", (2, 40, 5), np.nan),
                            ("B", (2, 40, 5), np.inf), ("scale", (2,), np.nan),
                            ("X", (4, 17), np.inf), ("X", (4, 17), np.nan), ("A", (2, 0, 0), -np.inf)):
        print(f"[adapters] {value} in {name}, tokens={tokens}", flush=True)
        bad = c[name].copy()
        bad[at] = value
        ids = c["adapter"].copy()
        ids[4] = 0
        y = _f64(_call(dq, dict(c, adapter=ids, **{name: bad})))
        hit = np.zeros((tokens, out), bool)
        if name == "X":
            hit[4] = True
        else:
            hit[ids == 2] = (np.arange(out) == 40) if name == "B" else True
        hit[4] |= ids[4] != c["adapter"][4]  # that token changed its adapter
        assert np.array_equal(y[~hit], clean[~hit])
        sure = hit.copy()
        sure[4] = hit[4] & (name == "X")
        assert not np.isfinite(y[sure]).any()


@pytest.mark.parametrize("tokens", [3, 200])
def test_rows_behind_the_last_token_and_the_workspace(dq, tokens):
    import torch

    c = _case(tokens, 1024, 96, 4, 16, seed=9)
    want = _call(dq, c)
    big = torch.full((tokens + 40, 96), 5.0, dtype=torch.bfloat16, device="cuda")
    need = dq.adapter_workspace_bytes(tokens, 1024, 16)
    space = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    y = _call(dq, c, y=big[:tokens], workspace=space[:need])
    assert torch.equal(y, want) and torch.all(big[tokens:] == 5.0) and torch.all(space[need:] == 77)


@pytest.mark.parametrize("tokens", [6, 300])
def test_streams_and_graph_replays(dq, tokens):
    import torch

    K, out, n, rank = 1024, 4128, 7, 24
    c = _case(tokens, K, out, n, rank, seed=10)
    X, adapter = _bf16(c["X"]), _dev(c["adapter"])
    A, B, scale, a = _bf16(c["A"]), _bf16(c["B"]), _dev(c["scale"]), _dev(c["a"])
    xc, xs = _dev(c["xc"]), _dev(c["xs"])
    pk = dq.gemm_pack_weights(_dev(c["wc"]), _dev(c["ws"]))
    y = torch.empty(tokens, out, dtype=torch.bfloat16, device="cuda")
    space = torch.empty(dq.adapter_workspace_bytes(tokens, K, rank), dtype=torch.uint8, device="cuda")
    call = lambda **k: dq.gemm_mx_adapters(xc, xs, pk, X, adapter, A, B, scale=scale, a=a, **k)  # noqa: E731
    call(y=y, workspace=space)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y=y, workspace=space)
    s = torch.cuda.Stream()
    for k in range(4):
        adapter.copy_(torch.randint(-1, n, (tokens,), device="cuda"))
        X.copy_(torch.randn(tokens, K, device="cuda"))
        y.zero_()
        g.replay()
        eager = call()
        s.wait_stream(torch.cuda.current_stream())
        other = call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(other, eager), k


def test_binding_refuses(dq):
    import torch

    c = _case(3, 512, 64, 2, 16)
    args = [_dev(c["xc"]), _dev(c["xs"]), dq.gemm_pack_weights(_dev(c["wc"]), _dev(c["ws"])),
            _bf16(c["X"]), _dev(c["adapter"]), _bf16(c["A"]), _bf16(c["B"])]
    assert dq.gemm_mx_adapters(*args).shape == (3, 64)
    X, ids, A, B = args[3:]
    bad = [{3: X.float()}, {3: X[:2]}, {3: X.cpu()}, {4: ids.long()}, {4: ids[:2]}, {4: ids[None]},
           {5: A[:, :, :256].contiguous()}, {5: A[0]}, {5: A.float()}, {5: A[:1]}, {6: B[:, :32].contiguous()},
           {6: B.transpose(1, 2).contiguous()}, {6: B.half()},
           {5: A[:, :4].contiguous(), 6: B[:, :, :4].contiguous()},
           {5: A.repeat(1, 17, 1), 6: B.repeat(1, 1, 17)}]
    for change in bad:
        with pytest.raises(ValueError):
            dq.gemm_mx_adapters(*[change.get(i, v) for i, v in enumerate(args)])
    for kw in (dict(scale=torch.ones(3, device="cuda")), dict(activation="swish"), dict(act_fmt="mxfp8"),
               dict(out_dtype="f16"), dict(bias=torch.ones(32, device="cuda")),
               dict(workspace=torch.zeros(8, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            dq.gemm_mx_adapters(*args, **kw)
    with pytest.raises(dq.DQError):
        dq.gemm_mx_adapters(*args, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
