"""The layer of experts on the GPU against a plain float64 implementation (layer_ref.moe), within
the bound that the products' arithmetic gives and the steps that the quantizer between them can
take within it."""
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


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _acts(tokens, K, fmt, seed):
    if fmt == "mxfp4":
        return workloads.mx_operands(tokens, K, seed=seed, lo=124, hi=130)
    return ref.mxfp8_operand(np.random.default_rng(seed), tokens, K)


def _experts(n, rows, K, seed, a=True):
    c, s = workloads.mx_operands(n * rows, K, seed=seed, lo=118, hi=124)
    v = None
    if a:
        v = np.random.default_rng(seed).uniform(0.1, 1.5, (n, rows)).astype(np.float32)
        v /= np.float32(np.sqrt(K))
    return c.reshape(n, rows, -1), s.reshape(n, rows, -1), v


def _pack(dq, w):
    return dq.gemm_pack_weights(_dev(w[0].reshape(-1, w[0].shape[2])),
                                _dev(w[1].reshape(-1, w[1].shape[2])))


def _flat(v):
    return None if v is None else _dev(v.reshape(-1))


def _layer(dq, n, K, inner, out, seed, a=True):
    gate, up = _experts(n, inner, K, seed + 1, a), _experts(n, inner, K, seed + 2, a)
    down = _experts(n, out, inner, seed + 3, a)
    b = np.random.default_rng(seed).uniform(0.5, 2.0, (n, inner)).astype(np.float32) if a else None
    return dict(gate=gate, up=up, down=down, b=b, n=n,
                dev=dict(gate=_pack(dq, gate), up=_pack(dq, up), down=_pack(dq, down), experts=n,
                         a_gate=_flat(gate[2]), a_up=_flat(up[2]), a_down=_flat(down[2]),
                         b_inner=_flat(b)))


def _routing(rng, tokens, n, top_k):
    ids = np.argsort(rng.standard_normal((tokens, n)) + rng.standard_normal(n), 1)[:, :top_k]
    return ids.astype(np.int32), rng.random((tokens, top_k)).astype(np.float32)


def _residual(rng, tokens, out, dtype):
    r = rng.standard_normal((tokens, out)).astype(np.float32)
    if dtype == "f32":
        return r, _dev(r)
    r = ref.bf16(r)
    return r, to_device((r.view(np.uint32) >> 16).astype(np.uint16), "bf16")


def _check(dq, L, xc, xs, ids, w, act_fmt="mxfp4", mid="mxfp8", dtype="bf16", kind="silu",
           residual=None, sample=None, **kw):
    y = dq.moe_mx(_dev(xc), _dev(xs), _dev(ids), _dev(w), activation=kind, act_fmt=act_fmt,
                  inner_fmt=mid, out_dtype=dtype, residual=None if residual is None else residual[1],
                  **L["dev"], **kw)
    r = None if residual is None else residual[0]
    ts = np.arange(len(ids)) if sample is None or len(ids) <= sample else np.unique(
        np.random.default_rng(1).choice(len(ids), sample))
    want, dy = layer_ref.moe(xc[ts], xs[ts], act_fmt, ids[ts], w[ts], L["gate"], L["up"], L["down"],
                             kind, L["b"], mid, None if r is None else r[ts])
    ref.check_rounded(_f64(y)[ts], want, dy, dtype)
    return y


# tokens, K, inner, out, experts, top_k: one token and many; every kernel of the selection (tiles of 32
# rows, of 64 where an expert has 3 rows or more and there are 340 tiles or where it has 40 and there are
# 128, or 256, of 128 from 129 rows and 256 tiles on); more pairs than a workgroup counts by itself; one
# expert; more experts than pairs
SHAPES = [(1, 512, 512, 512, 4, 2), (1, 1024, 512, 32, 64, 8), (3, 512, 1024, 96, 5, 3),
          (24, 512, 512, 160, 16, 4), (33, 1536, 512, 64, 2, 1), (40, 512, 512, 64, 3, 2),
          (61, 512, 1536, 288, 2, 2), (90, 512, 512, 64, 3, 2), (130, 1024, 512, 96, 2, 2),
          (200, 512, 512, 352, 1, 1), (300, 512, 512, 64, 12, 4), (700, 512, 512, 96, 6, 3),
          (45, 512, 512, 64, 40, 30), (200, 512, 1024, 1312, 64, 2), (130, 512, 1536, 1504, 32, 5),
          (700, 512, 1024, 1504, 4, 2), (4000, 512, 512, 1024, 2, 2), (3700, 512, 1024, 1120, 3, 3)]


@pytest.mark.parametrize("tokens,K,inner,out,n,top_k", SHAPES)
@pytest.mark.parametrize("act_fmt,mid,dtype", [("mxfp4", "mxfp8", "bf16"), ("mxfp4", "mxfp4", "f32"),
                                               ("mxfp8", "mxfp8", "bf16"), ("mxfp8", "mxfp4", "bf16")])
def test_shapes(dq, tokens, K, inner, out, n, top_k, act_fmt, mid, dtype):
    print(f"[moe] {tokens} x {K} -> {inner} -> {out}, {top_k} of {n}, {act_fmt} {mid} {dtype}",
          flush=True)
    rng = np.random.default_rng(tokens + n)
    L = _layer(dq, n, K, inner, out, 10 * n)
    xc, xs = _acts(tokens, K, act_fmt, tokens)
    ids, w = _routing(rng, tokens, n, top_k)
    _check(dq, L, xc, xs, ids, w, act_fmt, mid, dtype, residual=_residual(rng, tokens, out, dtype),
           sample=60)


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens", [4, 150])
def test_activations_and_optional_arrays(dq, kind, tokens):
    rng = np.random.default_rng(5)
    xc, xs = _acts(tokens, 512, "mxfp4", 6)
    ids, w = _routing(rng, tokens, 3, 2)
    for a in (True, False):
        print(f"[moe] {kind} tokens={tokens} a={a}", flush=True)
        L = _layer(dq, 3, 512, 512, 64, 7, a)
        _check(dq, L, xc, xs, ids, w, kind=kind, sample=40)


@pytest.mark.parametrize("tokens,n,top_k", [(3, 6, 2), (60, 2, 1), (300, 2, 2), (130, 64, 6)])
def test_8_bit_sums_are_whole(dq, tokens, n, top_k):
    # the values between the products show in what the down product makes of them: identity-like down
    # weights hand on one channel each, so a code that a truncated sum changed would be seen, step by
    # step. Outlier channels make the truncation of whole runs as large as it gets.
    K, inner, out = 2048, 512, 512
    rng = np.random.default_rng(tokens)
    x = rng.standard_normal((tokens, K))
    x[:, rng.random(K) < 0.02] *= 30.0
    xc, xs = ref.mxfp8(x.astype(np.float32), 32)
    L = _layer(dq, n, K, inner, out, 80, a=False)
    c, s = np.zeros((n, out, inner // 2), np.uint8), np.full((n, out, inner // 32), 127, np.uint8)
    for i in range(out):
        c[:, i, i // 2] = 2 << (4 * (i % 2))  # 1.0
    L["down"] = (c, s, None)
    L["dev"]["down"] = _pack(dq, L["down"])
    ids, _ = _routing(rng, tokens, n, top_k)
    w = np.zeros((tokens, top_k), np.float32)
    w[:, 0] = 1.0
    y = dq.moe_mx(_dev(xc), _dev(xs), _dev(ids), _dev(w), act_fmt="mxfp8", inner_fmt="mxfp4",
                  activation="relu", **L["dev"])
    wrong = total = 0
    for e in np.unique(ids[:, 0]):
        t = np.nonzero(ids[:, 0] == e)[0]
        one = lambda v: (v[0][e], v[1][e], None)  # noqa: E731
        h, dh = layer_ref.gated_whole(xc[t], xs[t], "mxfp8", one(L["gate"]), one(L["up"]), "relu")
        q, dq_ = layer_ref.quantized(h, dh, "mxfp4")
        got = _f64(y)[t]
        assert np.all(np.abs(got - q) <= dq_ + np.abs(q) * 2.0 ** -8)
        wrong += np.sum(np.abs(got - q) > np.abs(q) * 2.0 ** -8)
        total += q.size
    # only sums beside a border between two codes may go the other way
    assert wrong <= 1e-3 * total, (wrong, total)


@pytest.mark.parametrize("tokens", [1, 30, 400])
def test_ids_out_of_range_twice_and_all_alike(dq, tokens):
    n, K, inner, out, top_k = 5, 512, 512, 96, 4
    rng = np.random.default_rng(tokens)
    L = _layer(dq, n, K, inner, out, 20)
    xc, xs = _acts(tokens, K, "mxfp4", 21)
    w = rng.standard_normal((tokens, top_k)).astype(np.float32)
    res = _residual(rng, tokens, out, "bf16")
    for name, ids in dict(
            mixed=rng.choice([-1, 0, 1, 2, 3, 4, 5, 2 ** 31 - 1, -2 ** 31], (tokens, top_k)),
            alike=np.full((tokens, top_k), 3), twice=rng.choice([1, 4], (tokens, top_k)),
            none=np.full((tokens, top_k), -1)).items():
        print(f"[moe] ids {name} tokens={tokens}", flush=True)
        _check(dq, L, xc, xs, ids.astype(np.int32), w, residual=res, sample=40)
    y = _check(dq, L, xc, xs, np.full((tokens, top_k), n, np.int32), w, sample=40)
    assert float(y.abs().max()) == 0.0


@pytest.mark.parametrize("tokens", [12, 300])
@pytest.mark.parametrize("mid", ["mxfp4", "mxfp8"])
def test_nan_reaches_its_own_tokens_only(dq, tokens, mid):
    n, K, inner, out = 4, 512, 512, 64
    rng = np.random.default_rng(3)
    L = _layer(dq, n, K, inner, out, 30)
    xc, xs = _acts(tokens, K, "mxfp4", 31)
    ids, w = _routing(rng, tokens, n, 2)
    clean = _f64(_check(dq, L, xc, xs, ids, w, mid=mid, sample=40))
    xs = xs.copy()
    xs[5, 2] = 0xFF  # a token
    for name, row in (("gate", 7), ("down", 9)):
        print(f"[moe] nan in {name}, tokens={tokens}", flush=True)
        g = [v.copy() if v is not None else None for v in L[name]]
        g[1][2, row, 1] = 0xFF  # a row of expert 2
        y = _f64(dq.moe_mx(_dev(xc), _dev(xs), _dev(ids), _dev(w), inner_fmt=mid,
                           **{**L["dev"], name: _pack(dq, g)}))
        hit = (ids == 2).any(1)
        nan = np.zeros((tokens, out), bool)
        nan[hit] = True if name == "gate" else (np.arange(out) == row)[None]
        nan[5] = True
        assert np.array_equal(np.isnan(y), nan)
        assert np.array_equal(y[~nan], clean[~nan])


@pytest.mark.parametrize("tokens", [7, 260])
def test_in_place_and_rows_behind_the_last_token(dq, tokens):
    import torch

    n, K, inner, out = 6, 512, 512, 128
    rng = np.random.default_rng(8)
    L = _layer(dq, n, K, inner, out, 40)
    xc, xs = _acts(tokens, K, "mxfp4", 41)
    ids, w = _routing(rng, tokens, n, 3)
    for dtype, mid in (("bf16", "mxfp8"), ("f32", "mxfp4")):
        res = _residual(rng, tokens, out, dtype)
        want = _check(dq, L, xc, xs, ids, w, mid=mid, dtype=dtype, residual=res, sample=40)
        big = torch.full((tokens + 40, out), 5.0, device="cuda", dtype=want.dtype)
        y = big[:tokens]
        y.copy_(res[1])
        need = dq.moe_workspace_bytes(tokens, K, inner, out, n, 3)
        space = torch.full((need + 4096,), 77, device="cuda", dtype=torch.uint8)
        got = dq.moe_mx(_dev(xc), _dev(xs), _dev(ids), _dev(w), inner_fmt=mid, out_dtype=dtype,
                        residual=y, y=y, workspace=space[:need], **L["dev"])
        assert got is y and torch.equal(y, want)
        assert torch.all(big[tokens:] == 5.0) and torch.all(space[need:] == 77)


@pytest.mark.parametrize("tokens", [6, 400])
def test_streams_and_graph_replays(dq, tokens):
    # a graph reads the ids anew at every replay; eager work with its own workspace in between
    import torch

    n, K, inner, out, top_k = 9, 512, 512, 256, 3
    rng = np.random.default_rng(9)
    L = _layer(dq, n, K, inner, out, 50)
    xc, xs = (_dev(v) for v in _acts(tokens, K, "mxfp4", 51))
    ids = torch.zeros(tokens, top_k, dtype=torch.int32, device="cuda")
    w = torch.rand(tokens, top_k, device="cuda")
    y = torch.empty(tokens, out, dtype=torch.bfloat16, device="cuda")
    space = torch.empty(dq.moe_workspace_bytes(tokens, K, inner, out, n, top_k), dtype=torch.uint8,
                        device="cuda")
    call = lambda **k: dq.moe_mx(xc, xs, ids, w, **L["dev"], **k)  # noqa: E731
    call(y=y, workspace=space)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y=y, workspace=space)
    s = torch.cuda.Stream()
    for k in range(4):
        ids.copy_(_dev(_routing(rng, tokens, n, top_k)[0]))
        y.zero_()
        g.replay()
        eager = call()
        s.wait_stream(torch.cuda.current_stream())
        other = call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(other, eager), k


def test_calls_of_several_rounds(dq):
    # more tokens than one round's arrays hold (2^31 bytes of down products): equal tokens in every
    # round have equal results, and the first of them the definition's
    import torch

    n, K, inner, rows, out, top_k, tokens = 1, 512, 512, 4096, 1 << 19, 3, 400
    print(f"[moe] several rounds: {tokens} tokens, out {out}", flush=True)
    gate, up, down = _experts(n, inner, K, 61), _experts(n, inner, K, 62), _experts(n, rows, inner, 63)
    many = lambda v: _dev(v[0]).repeat(out // rows, 1)  # noqa: E731
    dev = dict(gate=_pack(dq, gate), up=_pack(dq, up), experts=n, a_gate=_flat(gate[2]),
               a_up=_flat(up[2]), a_down=_flat(down[2]).repeat(out // rows),
               down=dq.gemm_pack_weights(many(down[0]), many(down[1])))
    xc, xs = _acts(2, K, "mxfp4", 64)
    pick = np.arange(tokens) % 2
    ids = np.array([[0, 0, -1], [0, -1, -1]], np.int32)[pick]
    w = np.array([[0.5, 0.25, 9.0], [2.0, 9.0, 9.0]], np.float32)[pick]
    y = dq.moe_mx(_dev(xc[pick]), _dev(xs[pick]), _dev(ids), _dev(w), **dev)
    torch.cuda.synchronize()
    whole = y.view(tokens // 2, 2, out // rows, rows)
    assert torch.equal(whole, whole[:1, :, :1].expand_as(whole))
    want, dy = layer_ref.moe(xc, xs, "mxfp4", ids[:2], w[:2], gate, up, down, "silu", None, "mxfp8",
                             None)
    ref.check_rounded(_f64(y[:2, :rows]), want, dy, "bf16")


def test_binding_refuses(dq):
    import torch

    n, K, inner, out, tokens = 2, 512, 512, 64, 3
    L = _layer(dq, n, K, inner, out, 70)
    xc, xs = (_dev(v) for v in _acts(tokens, K, "mxfp4", 71))
    ids, w = (_dev(v) for v in _routing(np.random.default_rng(1), tokens, n, 2))
    ok = dict(L["dev"])
    assert dq.moe_mx(xc, xs, ids, w, **ok).shape == (tokens, out)
    bad = [dict(experts=3), dict(experts=0), dict(experts=4), dict(down=ok["gate"]),
           dict(up=dict(ok["up"], K=1024)), dict(a_gate=ok["a_gate"][1:]), dict(a_down=ok["a_gate"]),
           dict(b_inner=ok["b_inner"].double()), dict(activation="swish"), dict(inner_fmt="fp8"),
           dict(out_dtype="f16"), dict(residual=torch.zeros(tokens, out, device="cuda")),
           dict(y=torch.zeros(tokens, out + 1, dtype=torch.bfloat16, device="cuda")),
           dict(act_fmt="mxfp8"), dict(workspace=torch.zeros(8, dtype=torch.uint8)),
           dict(stream=torch.cuda.Stream(), gate=7)]
    for k, change in enumerate(bad):
        with pytest.raises(ValueError):
            dq.moe_mx(xc, xs, ids, w, **{**ok, **change})
            print("not refused:", k)
    for a in ((xc, xs, ids.long(), w), (xc, xs, ids, w.half()), (xc, xs, ids[:2], w[:2]),
              (xc, xs, ids, w[:, :1]), (xc, xs, ids.flatten(), w), (xc, xs, ids.cpu(), w),
              (xc, xs, ids.t().contiguous().t(), w)):
        with pytest.raises(ValueError):
            dq.moe_mx(*a, **ok)
    small = torch.zeros(dq.moe_workspace_bytes(tokens, K, inner, out, n, 2) - 256, dtype=torch.uint8,
                        device="cuda")
    for change in (dict(inner_fmt="nvfp4"), dict(out_dtype="f32"), dict(workspace=small),
                   dict(workspace=torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")[8:])):
        with pytest.raises(dq.DQError):
            dq.moe_mx(xc, xs, ids, w, **{**ok, **change})
    with pytest.raises(dq.DQError):
        dq.moe_mx(xc[:0], xs[:0], ids[:0], w[:0], **ok)
    with pytest.raises(dq.DQError):
        dq.moe_mx(xc, xs, ids.repeat(1, 17), w.repeat(1, 17), **ok)
