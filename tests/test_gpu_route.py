"""The router on the GPU against its definition in float64 (layer_ref.route): equal experts, and
weights within half a step of fp32 and the fp64 functions' own error."""
import numpy as np
import pytest

import layer_ref
import mlp_ref as ref

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


def _check_result(got, X, W, top_k, score="softmax", bias=None, renormalize=True, scale=1.0):
    ids, w = layer_ref.route(layer_ref.logits(X, W), top_k, score, bias, renormalize, scale)
    assert np.array_equal(got[0].cpu().numpy(), ids)
    g = got[1].cpu().numpy().astype(np.float64)
    # one rounding to fp32 (below its normal range half a step of 2^-149), and exp, sums and
    # quotients in fp64: well below 2^-40
    ok = np.abs(g - w) <= np.abs(w) * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -150
    assert np.all(ok | (np.isnan(g) & np.isnan(w))), (g[~ok][:4], w[~ok][:4])


def _check(dq, tokens, cols, experts, top_k, xdt="bf16", wdt="bf16", score="softmax", bias=False,
           renormalize=True, scale=1.0, seed=0):
    print(f"[route] {tokens}x{cols} {top_k} of {experts} {xdt}/{wdt} {score} bias={bias} "
          f"renormalize={renormalize} scale={scale}", flush=True)
    rng = np.random.default_rng(seed + tokens + experts)
    X = layer_ref.rounded(rng.standard_normal((tokens, cols)).astype(np.float32), xdt)
    W = layer_ref.rounded((rng.standard_normal((experts, cols)) * 1.5 / np.sqrt(cols)).astype(
        np.float32), wdt)
    b = (0.2 * rng.standard_normal(experts)).astype(np.float32) if bias else None
    got = dq.moe_route(_tensor(X, xdt), _tensor(W, wdt), top_k, score=score, bias=_tensor(b),
                       renormalize=renormalize, scale=scale)
    _check_result(got, X, W, top_k, score, b, renormalize, np.float32(scale).astype(np.float64))


@pytest.mark.parametrize("tokens,cols,experts,top_k", [
    (1, 8, 1, 1), (1, 4096, 64, 8), (1, 520, 257, 32), (2, 1000, 63, 5), (3, 512, 65, 8),
    (5, 2048, 128, 4), (17, 128, 1024, 32), (33, 8, 7, 7), (64, 1536, 129, 6), (65, 4096, 64, 8),
    (70, 24, 5, 2), (97, 1000, 33, 3), (256, 520, 256, 8), (1000, 264, 100, 1), (130, 40, 1024, 32),
    (2100, 1000, 130, 8), (1111, 520, 520, 5), (33000, 8, 1024, 4), (3000, 1032, 129, 8),
    (1000, 4104, 70, 5), (700, 2104, 200, 6), (16, 4096, 1024, 4), (2, 65536, 100, 3),
    (20, 65536, 1000, 2), (66, 8200, 1000, 7), (300, 520, 130, 4), (900, 264, 150, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_shapes(dq, tokens, cols, experts, top_k, score):
    _check(dq, tokens, cols, experts, top_k, score=score, bias=tokens % 2 == 1)


@pytest.mark.parametrize("xdt", ["bf16", "f32"])
@pytest.mark.parametrize("wdt", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 9, 200, 4000])
def test_types_and_weights(dq, xdt, wdt, tokens):
    for k, (score, bias, renormalize, scale) in enumerate((
            ("softmax", False, True, 1.0), ("softmax", True, False, 2.5),
            ("sigmoid", True, True, 2.5), ("sigmoid", False, False, -0.1))):
        _check(dq, tokens, 776, 96, 6, xdt, wdt, score, bias, renormalize, scale, seed=k)


@pytest.mark.parametrize("tokens", [4, 100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(dq, tokens, score):
    # equal experts, and tokens of zeros (every logit 0)
    rng = np.random.default_rng(3)
    X = ref.bf16(rng.standard_normal((tokens, 256)).astype(np.float32))
    X[1] = 0.0
    W = ref.bf16(rng.standard_normal((150, 256)).astype(np.float32) / 16)
    W = W[rng.integers(0, 40, 150)]
    for top_k in (1, 7, 32):
        got = dq.moe_route(_tensor(X, "bf16"), _tensor(W, "bf16"), top_k, score=score)
        _check_result(got, X, W, top_k, score)
        assert np.array_equal(got[0][1].cpu().numpy(), np.arange(top_k))


@pytest.mark.parametrize("tokens", [3, 90])
def test_close_logits_do_not_depend_on_the_order_of_a_sum(dq, tokens):
    # experts whose logits differ by about an fp32 step, of sums that cancel
    rng = np.random.default_rng(4)
    cols, n = 2048, 64
    X = ref.bf16(rng.standard_normal((tokens, cols)).astype(np.float32) * 30)
    W = np.repeat(rng.standard_normal((1, cols)).astype(np.float32), n, 0)
    W[:, 0] += rng.standard_normal(n).astype(np.float32) * 1e-6
    got = dq.moe_route(_tensor(X, "bf16"), _tensor(W), 8, score="softmax")
    _check_result(got, X, W, 8)


def test_extreme_and_non_finite_values(dq):
    import torch

    cols, n = 64, 10
    rng = np.random.default_rng(5)
    W = rng.standard_normal((n, cols)).astype(np.float32)
    X = np.zeros((8, cols), np.float32)
    X[0] = rng.standard_normal(cols) * 1e4    # one score 1, the others 0
    X[1] = -W[0] * 1e3
    X[2] = np.nan
    X[3, 0] = np.inf
    X[4] = 1e-40
    X[5] = rng.standard_normal(cols) * 3e37   # logits may overflow fp32
    for score in ("softmax", "sigmoid"):
        got = dq.moe_route(_tensor(X), _tensor(W), 4, score=score)
        ids = got[0].cpu().numpy()
        assert np.all((ids >= 0) & (ids < n)) and all(len(set(r)) == 4 for r in ids.tolist())
        rows = [0, 1, 4, 6, 7]
        _check_result([g[rows] for g in got], X[rows], W, 4, score)
        assert np.array_equal(ids[2], np.arange(4)) and torch.isnan(got[1][2]).all()
    # every score zero: zero weights, no quotient of zeros
    X = -1e6 * np.ones((1, cols), np.float32)
    got = dq.moe_route(_tensor(X), _tensor(np.ones((n, cols), np.float32)), 3, score="sigmoid")
    assert float(got[1].abs().max()) == 0.0 and got[0].tolist() == [[0, 1, 2]]
    # a bias alone decides where the scores agree; infinities and a NaN in it
    b = np.array([0, 1, np.inf, -np.inf, np.nan, 2, 1, 0, 0, 0], np.float32)
    got = dq.moe_route(_tensor(np.zeros((1, cols), np.float32)), _tensor(W), 10, bias=_tensor(b))
    assert got[0].tolist() == [[2, 5, 1, 6, 0, 7, 8, 9, 3, 4]]


@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("tokens,cols,experts,top_k", [
    (150, 64, 40, 8), (700, 2048, 200, 8), (1100, 2048, 130, 32), (600, 4096, 130, 8),
    (690, 448, 1024, 5), (2100, 8192, 33, 1), (1500, 4096, 50, 4), (3000, 2560, 129, 32)])
def test_many_tokens_close_logits(dq, tokens, cols, experts, top_k, score, bias):
    # sums of large terms that cancel, and experts that differ in the last bit of a few weights: far
    # more of them in question than are chosen (large products go by bounds, those of up to 1024 tokens
    # with four waves a token)
    rng = np.random.default_rng(cols + experts)
    X = ref.bf16(rng.standard_normal((tokens, cols)).astype(np.float32) * 8)
    W = ref.bf16(rng.standard_normal((experts // 8 + 1, cols)).astype(np.float32))
    W = W[rng.integers(0, len(W), experts)].copy()
    at = rng.integers(0, cols, (experts, 2))
    bits = W.view(np.uint32)
    for k in range(2):
        bits[np.arange(experts), at[:, k]] ^= rng.integers(0, 2, experts).astype(np.uint32) << 16
    X *= 2.0 ** -np.round(np.log2(np.sqrt(cols)))
    b = (rng.integers(0, 3, experts) * 0.25).astype(np.float32) if bias else None
    got = dq.moe_route(_tensor(X, "bf16"), _tensor(W, "bf16"), top_k, score=score, bias=_tensor(b),
                       scale=2.0)
    _check_result(got, X, W, top_k, score, b, True, 2.0)


@pytest.mark.parametrize("tokens", [600, 1100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens_numbers_of_experts_in_question(dq, score, tokens):
    # n experts that are alike and above all others: that many are in question, in several registers of
    # a wave from 65 on; ties go to the lowest, scattered as they lie
    cols, experts, top_k = 2304, 200, 8
    rng = np.random.default_rng(tokens)
    X = ref.bf16(rng.standard_normal((tokens, cols)).astype(np.float32))
    X[:, 0] = 4.0
    for n in (8, 9, 15, 16, 17, 63, 64, 65, 72, 129, 200):
        W = ref.bf16((rng.standard_normal((experts, cols)) / 64).astype(np.float32))
        alike = np.sort(rng.permutation(experts)[:n])
        W[alike] = W[alike[0]]
        W[alike, 0], W[np.setdiff1d(np.arange(experts), alike), 0] = 2.0, -2.0
        print(f"[route] {n} in question", flush=True)
        got = dq.moe_route(_tensor(X, "bf16"), _tensor(W, "bf16"), top_k, score=score)
        assert np.array_equal(got[0].cpu().numpy(), np.tile(alike[:top_k], (tokens, 1)))
        _check_result(got, X, W, top_k, score)


@pytest.mark.parametrize("tokens", [600, 1100])
def test_many_tokens_wide_scores_and_biases(dq, tokens):
    # logits from -900 to 900: scores down to the smallest fp64 values and ties at 0 and 1; biases
    # beyond fp32's resolution of the scores, of both signs, infinite and NaN
    cols, experts, top_k = 2304, 200, 12
    rng = np.random.default_rng(tokens + 1)
    X = ref.bf16(rng.standard_normal((tokens, cols)).astype(np.float32))
    W = ref.bf16((rng.standard_normal((experts, cols)) * 4).astype(np.float32))
    X *= np.exp2(rng.integers(-12, 2, (tokens, 1))).astype(np.float32)
    X[:40] = -np.abs(X[:40])
    W[:, :512] = np.abs(W[:, :512])
    b = (rng.standard_normal(experts) * 10.0 ** rng.integers(-9, 3, experts)).astype(np.float32)
    b[[3, 50, 120, 199]] = [np.inf, -np.inf, np.nan, 1e38]
    for bias in (None, b):
        print(f"[route] wide, bias {bias is not None}", flush=True)
        got = dq.moe_route(_tensor(X, "bf16"), _tensor(W, "bf16"), top_k, score="sigmoid",
                           bias=_tensor(bias))
        _check_result(got, X, W, top_k, "sigmoid", bias)


@pytest.mark.parametrize("tokens", [100, 1000, 1030])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens_non_finite_and_extreme_values(dq, score, tokens):
    rng = np.random.default_rng(8)
    cols, n = 4096, 70
    W = ref.bf16(rng.standard_normal((n, cols)).astype(np.float32))
    X = ref.bf16(rng.standard_normal((tokens, cols)).astype(np.float32))
    X[3], X[4, 7], X[5, 9], X[6] = 0, np.nan, np.inf, X[6] * np.float32(2 ** 100)
    X[7], X[8], X[9] = X[7] * np.float32(2 ** 124), X[8] * np.float32(2 ** -130), X[9] * np.float32(2 ** 12)
    X[8] = ref.bf16(X[8])  # subnormal there
    for change in ("none", "nan", "inf", "huge"):
        V = W.copy()
        if change != "none":
            V[50, 3] = dict(nan=np.nan, inf=-np.inf, huge=np.float32(2 ** 126))[change]
        print(f"[route] many tokens, {score}, {change}", flush=True)
        with np.errstate(all="ignore"):
            got = dq.moe_route(_tensor(X, "bf16"), _tensor(V, "bf16"), 6, score=score)
            # rows whose sums have several infinities or NaN depend on nothing here: NaN or not is
            # the definition's in every row, and so are the experts
            _check_result(got, X, V, 6, score)


@pytest.mark.parametrize("tokens", [6, 130, 6600, 13200])
def test_given_arrays_streams_and_graph_replays(dq, tokens):
    import torch

    X = torch.randn(tokens, 512, device="cuda").to(torch.bfloat16)
    W = torch.randn(40, 512, device="cuda").to(torch.bfloat16)
    ids = torch.full((tokens + 3, 5), 99, dtype=torch.int32, device="cuda")
    w = torch.full((tokens + 3, 5), 99.0, device="cuda")
    need = dq.moe_route_workspace_bytes(tokens, 40)
    space = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
    call = lambda **k: dq.moe_route(X, W, 5, **k)  # noqa: E731
    given = dict(ids=ids[:tokens], weights=w[:tokens], workspace=space[:need])
    got = call(**given)
    assert got[0] is given["ids"] and got[1] is given["weights"]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(**given)
    s = torch.cuda.Stream()
    for k in range(4):
        X.copy_(torch.randn(tokens, 512, device="cuda"))
        g.replay()
        eager = call()
        s.wait_stream(torch.cuda.current_stream())
        other = call(stream=s)
        torch.cuda.synchronize()
        for a, b, c in zip(got, eager, other):
            assert torch.equal(a, b) and torch.equal(a, c), k
    assert torch.all(ids[tokens:] == 99) and torch.all(w[tokens:] == 99) and torch.all(space[need:] == 7)


def test_binding_refuses(dq):
    import torch

    X, W = torch.randn(3, 64, device="cuda"), torch.randn(6, 64, device="cuda")
    for a, kw in (((X, W, 0), {}), ((X, W, 7), {}), ((X, W, 33), {}), ((X.half(), W, 2), {}),
                  ((X, W.double(), 2), {}), ((X, W[:, :32], 2), {}), ((X.t(), W, 2), {}),
                  ((X, W.cpu(), 2), {}), ((X.cpu(), W, 2), {}), ((X[0], W, 2), {}),
                  ((X, W, 2), dict(score="max")), ((X, W, 2), dict(bias=torch.ones(5, device="cuda"))),
                  ((X, W, 2), dict(ids=torch.zeros(3, 2, device="cuda"))),
                  ((X, W, 2), dict(weights=torch.zeros(3, 3, device="cuda"))),
                  ((X, W, 2), dict(workspace=torch.zeros(512, dtype=torch.uint8)))):
        with pytest.raises(ValueError):
            dq.moe_route(*a, **kw)
    for a, kw in (((X[:, :12].contiguous(), W[:, :12].contiguous(), 2), {}), ((X[:0], W, 2), {}),
                  ((X, W, 2), dict(scale=float("inf"))),
                  ((X, W, 2), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(dq.DQError):
            dq.moe_route(*a, **kw)
