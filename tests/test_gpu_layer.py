"""The operators of include/dq_layer.h together, as a decoder layer with experts runs them: norm after
the attention and before the experts, router, experts onto the residual stream, norm after the experts
and before the next projection, that projection with each request's adapter. Every step is checked
against its definition on the values that the step before left on the GPU."""
import numpy as np
import pytest

import layer_ref
import mlp_ref as ref
import workloads
from parity import host

pytestmark = pytest.mark.gpu

H, I, E, TOP, OUT, RANK, ADAPTERS = 1024, 512, 12, 3, 1280, 16, 5


@pytest.fixture(scope="module")
def dq():
    import torch

    assert torch.cuda.is_available()
    import dual_scale_w4a4_amd

    dual_scale_w4a4_amd.lib()
    return dual_scale_w4a4_amd


def _dev(a, dtype="f32"):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def _np(t):
    return t.float().cpu().numpy()


class Layer:
    def __init__(self, dq, seed=0):
        self.dq, rng = dq, np.random.default_rng(seed)
        f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731

        def weights(n, rows, K, k):
            c, s = workloads.mx_operands(n * rows, K, seed=seed + k, lo=118, hi=122)
            a = (rng.uniform(0.2, 1.0, (n, rows)) / np.sqrt(K) * 8).astype(np.float32)
            return c.reshape(n, rows, -1), s.reshape(n, rows, -1), a

        self.gate, self.up, self.down = weights(E, I, H, 1), weights(E, I, H, 2), weights(E, H, I, 3)
        self.proj = weights(1, OUT, H, 4)
        self.w = {k: layer_ref.rounded(1 + 0.1 * f(H), "bf16") for k in ("post1", "pre1", "post2", "pre2")}
        self.gates = np.tanh(f(H))
        self.b = np.ldexp(np.float32(1), rng.integers(-1, 2, H)).astype(np.float32)
        self.router = layer_ref.rounded(f(E, H) / 16, "bf16")
        self.A = layer_ref.rounded(f(ADAPTERS, RANK, H) / 32, "bf16")
        self.B = layer_ref.rounded(f(ADAPTERS, OUT, RANK), "bf16")
        pack = lambda w: dq.gemm_pack_weights(*(_dev(v.reshape(-1, v.shape[2])) for v in w[:2]))  # noqa: E731
        self.d = dict(gate=pack(self.gate), up=pack(self.up), down=pack(self.down), proj=pack(self.proj),
                      ag=_dev(self.gate[2].reshape(-1)), au=_dev(self.up[2].reshape(-1)),
                      ad=_dev(self.down[2].reshape(-1)), ap=_dev(self.proj[2].reshape(-1)),
                      b=_dev(self.b), gates=_dev(self.gates), router=_dev(self.router, "bf16"),
                      A=_dev(self.A, "bf16"), B=_dev(self.B, "bf16"),
                      **{k: _dev(v, "bf16") for k, v in self.w.items()})

    def buffers(self, tokens):
        import torch

        o = {}
        e = lambda name, shape, dt: o.__setitem__(name, torch.zeros(shape, dtype=dt, device="cuda"))  # noqa: E731
        for n in ("1", "2"):
            e("codes" + n, (tokens, H // 2), torch.uint8)
            e("scales" + n, (tokens, H // 32), torch.uint8)
            e("h" + n, (tokens, H), torch.bfloat16)
            e("x" + n, (tokens, H), torch.bfloat16)
        e("ids", (tokens, TOP), torch.int32)
        e("weights", (tokens, TOP), torch.float32)
        e("y", (tokens, H), torch.bfloat16)
        e("out", (tokens, OUT), torch.bfloat16)
        e("status", (1,), torch.int32)
        dq = self.dq
        for name, n in (("space1", dq.moe_route_workspace_bytes(tokens, E)),
                        ("space2", dq.moe_workspace_bytes(tokens, H, I, H, E, TOP)),
                        ("space3", dq.adapter_workspace_bytes(tokens, H, RANK))):
            e(name, (n,), torch.uint8)
        return o

    def run(self, attn, stream_in, adapter, o, **kw):
        dq, d = self.dq, self.d
        dq.block_norm_quantize_act_async(attn, "mxfp4", 32, o["codes1"], o["scales1"], o["status"],
                                         residual=stream_in, residual_out=o["h1"], x_out=o["x1"],
                                         post_weight=d["post1"], weight=d["pre1"], b=d["b"],
                                         residual_scale=0.75, **kw)
        dq.moe_route(o["x1"], d["router"], TOP, score="sigmoid", scale=1.5, ids=o["ids"],
                     weights=o["weights"], workspace=o["space1"], **kw)
        dq.moe_mx(o["codes1"], o["scales1"], o["ids"], o["weights"], d["gate"], d["up"], d["down"], E,
                  a_gate=d["ag"], a_up=d["au"], a_down=d["ad"], y=o["y"], workspace=o["space2"], **kw)
        dq.block_norm_quantize_act_async(o["y"], "mxfp4", 32, o["codes2"], o["scales2"], o["status"],
                                         residual=o["h1"], residual_out=o["h2"], x_out=o["x2"],
                                         post_weight=d["post2"], gate=d["gates"], weight=d["pre2"],
                                         b=d["b"], **kw)
        dq.gemm_mx_adapters(o["codes2"], o["scales2"], d["proj"], o["x2"], adapter, d["A"], d["B"],
                            a=d["ap"], y=o["out"], workspace=o["space3"], **kw)


def _inputs(tokens, seed):
    rng = np.random.default_rng(seed)
    f = lambda: layer_ref.rounded(rng.standard_normal((tokens, H)).astype(np.float32), "bf16")  # noqa: E731
    return f(), f(), rng.integers(-1, ADAPTERS, tokens).astype(np.int32)


@pytest.mark.parametrize("tokens", [1, 7, 33, 130])
def test_every_step_of_a_layer(dq, oracle_lib, tokens):
    import torch

    L = Layer(dq)
    attn, R, adapter = _inputs(tokens, tokens)
    o = L.buffers(tokens)
    L.run(_dev(attn, "bf16"), _dev(R, "bf16"), _dev(adapter), o)
    torch.cuda.synchronize()
    assert int(o["status"].item()) == 0

    def norm(X, res, n, gate, rs, post, pre):
        h, v, x = layer_ref.block_norm(X, res, L.w[post], gate, None, rs, L.w[pre], L.b, "bf16")
        q = oracle_lib.quantize_act(x, "f32", "mxfp4", 32, None, 0.0)
        assert np.array_equal(_np(o["h" + n]), h) and np.array_equal(_np(o["x" + n]), ref.bf16(v))
        assert np.array_equal(host(o["codes" + n]), q["codes"])
        assert np.array_equal(host(o["scales" + n]), q["scales"])

    norm(attn, R, "1", None, 0.75, "post1", "pre1")
    ids, w = layer_ref.route(layer_ref.logits(_np(o["x1"]), L.router), TOP, "sigmoid", None, True, 1.5)
    assert np.array_equal(host(o["ids"]), ids)
    assert np.all(np.abs(host(o["weights"]) - w) <= np.abs(w) * (2.0 ** -24 + 2.0 ** -40))
    y, dy = layer_ref.moe(host(o["codes1"]), host(o["scales1"]), "mxfp4", ids, host(o["weights"]),
                          L.gate, L.up, L.down, "silu", None, "mxfp8", None)
    ref.check_rounded(_np(o["y"]).astype(np.float64), y, dy, "bf16")
    norm(_np(o["y"]), _np(o["h1"]), "2", L.gates, 1.0, "post2", "pre2")
    y, dy = layer_ref.adapters(host(o["codes2"]), host(o["scales2"]), "mxfp4", *(v[0] for v in L.proj),
                               None, "none", None, _np(o["x2"]), adapter, L.A, L.B, None, "bf16")
    ref.check_rounded(_np(o["out"]).astype(np.float64), y, dy, "bf16")


@pytest.mark.parametrize("tokens", [2, 90])
def test_a_captured_layer_beside_eager_ones(dq, tokens):
    # one graph replayed on new inputs, with eager runs on two streams and other arrays in between
    import torch

    L = Layer(dq, 3)
    ins = [t for t in (_dev(v, "bf16" if k < 2 else "f32") for k, v in enumerate(_inputs(tokens, 1)))]
    graphed, eager, side = (L.buffers(tokens) for _ in range(3))
    L.run(*ins, graphed)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.run(*ins, graphed)
    s = torch.cuda.Stream()
    for k in range(4):
        for t, v in zip(ins, _inputs(tokens, 10 + k)):
            t.copy_(_dev(v))
        for o in (graphed, eager, side):
            for n in ("out", "y", "ids", "h2"):
                o[n].zero_()
        g.replay()
        s.wait_stream(torch.cuda.current_stream())
        L.run(*ins, side, stream=s)
        L.run(*ins, eager)
        torch.cuda.synchronize()
        for n in ("out", "y", "ids", "weights", "h1", "h2", "codes2", "scales2", "x2"):
            assert torch.equal(graphed[n], eager[n]) and torch.equal(side[n], eager[n]), (k, n)


def test_two_threads_at_once(dq):
    import threading

    import torch

    L = Layer(dq, 5)
    sets = []
    for k in range(2):
        attn, R, ids = _inputs(20, 40 + k)
        ins = _dev(attn, "bf16"), _dev(R, "bf16"), _dev(ids)
        want, o = L.buffers(20), L.buffers(20)
        L.run(*ins, want)
        sets.append((ins, want, o))
    torch.cuda.synchronize()
    bad = []

    def work(ins, want, o):
        s = torch.cuda.Stream()
        for _ in range(20):
            o["out"].zero_()
            s.wait_stream(torch.cuda.current_stream())
            L.run(*ins, o, stream=s)
            s.synchronize()
            bad.append(not torch.equal(o["out"], want["out"]))

    ts = [threading.Thread(target=work, args=a) for a in sets]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert len(bad) == 40 and not any(bad)
