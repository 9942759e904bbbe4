"""Cases of the operators for decoder layers with experts, adapters and norms on both sides of
their blocks, for timing and comparison.

  norm      the norms after one block and before the next, with the block's gate and the
            residual's scale between them:
              m = (X r1) post_j gate_j tgate_t,  r1 = 1 / sqrt(mean X^2 + eps)  (m = X .. without
              a post norm);  h = residual_scale residual + m, stored in X's type;
              n = (h r2) weight_j, stored as well where asked for;  x = n b_j, quantized to MXFP8;
  route     the experts of each token: the top_k largest scores (softmax or sigmoid of X W^T, a
            bias per expert added for the selection only), and their weights;
  moe       a layer of experts: the gated product, the quantizer (MXFP8) and the down product of
            each token's experts, summed with the tokens' weights onto a residual;
  adapter   Y = residual + act(a_i sum_k x^ Qhat + bias_i + scale_r sum_j (sum_k X A_r) B_r), the
            product with MXFP4 weights that all requests share and each token's low-rank adapter r.

`run` computes them with elementary torch operations in fp32 (the router's scores, which are next
to each other, in float64), or, where `own` is true, with this package's kernels. `exact` evaluates
the same definitions in float64.

Sizes are the MLP shapes this repository solves (hidden 4096, inner 14336) and generic ones.
"""
import math

import torch

own = False

GROUP = 32
EPS = 1e-5


def listed():
    H, I = 4096, 14336
    return [
        # between the attention and the MLP of one decoding sequence: latency
        dict(name="norm one token", op="norm", tokens=1, cols=H, dtype="bf16", post=True,
             gate=False, token_gate=False, x_out=True),
        # the same for a prompt, with a gate per channel: memory bandwidth
        dict(name="norm prompt", op="norm", tokens=8192, cols=H, dtype="bf16", post=True,
             gate=True, token_gate=False, x_out=True),
        # an fp32 stream, a gate per token, no post norm, a width that is no multiple of a tile
        dict(name="norm ragged fp32", op="norm", tokens=1003, cols=8160, dtype="f32", post=False,
             gate=False, token_gate=True, x_out=False),
        # the router of one decoding sequence: latency
        dict(name="route one token", op="route", tokens=1, cols=H, experts=64, top_k=8,
             dtype="bf16", score="softmax", bias=False),
        # the router of a prompt, with sigmoid scores and a balancing bias
        dict(name="route prompt", op="route", tokens=4096, cols=H, experts=128, top_k=8,
             dtype="bf16", score="sigmoid", bias=True),
        # a layer of small experts for one decoding sequence: reads 8 experts' weights
        dict(name="moe one token", op="moe", tokens=1, K=2048, inner=1024, experts=64, top_k=8,
             act_fmt="mxfp4", act="silu", residual=True),
        # 24 sequences decoding together: nearly every expert's weights, a few tokens each
        dict(name="moe 24 sequences", op="moe", tokens=24, K=H, inner=1536, experts=64, top_k=8,
             act_fmt="mxfp4", act="silu", residual=True),
        # few large experts, 8-bit activations, an odd number of sequences
        dict(name="moe 8-bit 5 sequences", op="moe", tokens=5, K=H, inner=I, experts=8, top_k=2,
             act_fmt="mxfp8", act="silu", residual=False),
        # a chunk of a prompt: about 90 tokens an expert
        dict(name="moe chunk of a prompt", op="moe", tokens=700, K=H, inner=1536, experts=32,
             top_k=4, act_fmt="mxfp4", act="gelu_tanh", residual=True),
        # the down projection of 32 sequences decoding together, nearly each with its own adapter
        dict(name="adapter 32 sequences", op="adapter", tokens=32, K=I, out=H, rank=16,
             adapters=40, packed=False, act_fmt="mxfp4", dtype="bf16", bias=False, act="none",
             residual=True),
        # prompts of several requests packed into one batch
        dict(name="adapter prompts", op="adapter", tokens=4096, K=H, out=I, rank=64, adapters=6,
             packed=True, act_fmt="mxfp4", dtype="bf16", bias=False, act="none", residual=False),
        # odd sizes, bias and activation, fp32 out
        dict(name="adapter ragged", op="adapter", tokens=515, K=2560, out=1733, rank=24,
             adapters=5, packed=True, act_fmt="mxfp4", dtype="f32", bias=True, act="gelu_tanh",
             residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "route", "moe", "moe", "adapter", "adapter"))
    if op == "norm":
        c = dict(op=op, tokens=_log(rng, 1, 8192), cols=32 * _log(rng, 16, 448),
                 dtype=rng.choice(("bf16", "f32")), post=rng.random() < 0.7,
                 gate=rng.random() < 0.4, token_gate=rng.random() < 0.3, x_out=rng.random() < 0.6)
        while c["tokens"] * c["cols"] * (2 if c["dtype"] == "f32" else 1) > 8192 * 4096:
            c["tokens"] //= 2
        return c
    if op == "route":
        c = dict(op=op, tokens=_log(rng, 1, 4096), cols=32 * _log(rng, 16, 256),
                 experts=_log(rng, 8, 256), dtype=rng.choice(("bf16", "f32")),
                 score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5)
        c["top_k"] = rng.randint(1, min(8, c["experts"]))
        while c["tokens"] * c["cols"] * c["experts"] > 4096 * 4096 * 128:
            c["tokens"] //= 2
        return c
    act_fmt = rng.choice(("mxfp4", "mxfp8"))
    if op == "moe":
        c = dict(op=op, tokens=_log(rng, 1, 700), K=512 * _log(rng, 1, 12),
                 inner=512 * _log(rng, 1, 28), experts=_log(rng, 4, 128), act_fmt=act_fmt,
                 act=rng.choice(("silu", "gelu_tanh")), residual=rng.random() < 0.5)
        c["top_k"] = rng.randint(1, min(8, c["experts"]))
        while c["experts"] * c["K"] * c["inner"] > 8 * 4096 * 14336:
            c["inner"] = max(512, c["inner"] // 1024 * 512)
            if c["inner"] == 512:
                c["K"] = max(512, c["K"] // 1024 * 512)
        while c["tokens"] * c["experts"] * c["K"] * c["inner"] > 700 * 32 * 4096 * 1536:
            c["tokens"] //= 2
        return c
    c = dict(op=op, tokens=_log(rng, 1, 4096), K=512 * _log(rng, 1, 28), out=_log(rng, 40, 14336),
             rank=8 * _log(rng, 1, 16), adapters=_log(rng, 1, 48), packed=rng.random() < 0.5,
             act_fmt=act_fmt, dtype=rng.choice(("bf16", "f32")) if act_fmt == "mxfp4" else "bf16",
             bias=rng.random() < 0.4, act=rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")),
             residual=rng.random() < 0.6)
    while c["tokens"] * (c["K"] * c["out"] + c["adapters"] * c["rank"] * (c["K"] + c["out"])) > (
            4096 * (4096 * 14336 + 6 * 64 * (4096 + 14336))):
        c["tokens"] //= 2
    return c


# ------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _stream(g, tokens, cols):
    """Rows of a hidden-state stream: N(0, 1) times a level per channel, a few channels larger."""
    level = torch.exp(0.5 * _randn(g, cols))
    big = torch.rand(cols, device="cuda", generator=g) < 0.01
    return _randn(g, tokens, cols) * torch.where(big, level * 20.0, level)


def _pow2(g, n, lo, hi):
    """Powers of two 2^lo .. 2^hi: values of every outer scale set."""
    return torch.exp2(torch.randint(lo, hi + 1, (n,), device="cuda", generator=g).float())


def _weights(g, out, K):
    """MXFP4 weights as the solver leaves them: codes (out x K/2), E8M0 bytes (out x K/32), row
    scales a, and the codes and scales laid out for the packed product. Experts' weights are one
    such matrix, their rows one expert after the other."""
    e, v = _quantize_values(_randn(g, out, K) * (1.0 / math.sqrt(K)), "mxfp4")
    codes, scales = _fp4_codes(v), (e + 127).to(torch.uint8)
    del e, v
    nrb, nst = -(-out // 32), K // 256
    pc = torch.zeros(nrb * 32, K // 2, dtype=torch.uint8, device="cuda")
    ps = torch.full((nrb * 32, K // 32), 127, dtype=torch.uint8, device="cuda")
    pc[:out], ps[:out] = codes, scales
    pc = pc.view(nrb, 32, nst, 2, 4, 16).permute(0, 2, 4, 3, 1, 5).contiguous().view(-1)
    ps = ps.view(nrb, 32, nst, 2, 4).permute(0, 2, 3, 1, 4).contiguous().view(-1)
    return dict(codes=codes, scales=scales, a=_pow2(g, out, -1, 1),
                packed=dict(codes=pc, scales=ps, out=out, K=K))


def _activations(x, fmt):
    e, v = _quantize_values(x, fmt)
    return (_fp4_codes(v) if fmt == "mxfp4" else _fp8_codes(v)), (e + 127).to(torch.uint8)


def _requests(g, case):
    """Each token's adapter, -1 for none: a decoding sequence's own, or a few prompts one after
    the other."""
    t, n = case["tokens"], case["adapters"]
    if not case["packed"]:
        return torch.randint(-1, n, (t,), device="cuda", generator=g, dtype=torch.int32)
    edges = torch.sort(torch.randint(0, t + 1, (n,), device="cuda", generator=g)).values
    of = torch.searchsorted(edges, torch.arange(t, device="cuda"), right=True)
    which = torch.randint(-1, n, (n + 1,), device="cuda", generator=g, dtype=torch.int32)
    return which[of].contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, tokens = case["op"], case["tokens"]
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    s = dict(case=case)
    if op == "norm":
        n = case["cols"]
        s["X"] = _stream(g, tokens, n).to(dt)
        s["residual"] = _stream(g, tokens, n).to(dt)
        s["post"] = (1.0 + 0.2 * _randn(g, n)).to(dt) if case["post"] else None
        s["weight"] = (1.0 + 0.2 * _randn(g, n)).to(dt)
        s["gate"] = torch.tanh(_randn(g, n)) if case["gate"] else None
        s["token_gate"] = torch.sigmoid(_randn(g, tokens)) if case["token_gate"] else None
        s["residual_scale"] = 0.75
        s["b"] = _pow2(g, n, -3, 3)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    if op == "route":
        n, e = case["cols"], case["experts"]
        s["X"] = _randn(g, tokens, n).to(dt)
        s["W"] = (_randn(g, e, n) * (1.5 / math.sqrt(n))).to(dt)
        s["bias"] = 0.1 * _randn(g, e) if case["bias"] else None
        return s
    K = case["K"]
    if op == "moe":
        e, inner = case["experts"], case["inner"]
        s["codes"], s["scales"] = _activations(_stream(g, tokens, K), case["act_fmt"])
        logits = _randn(g, tokens, e) + 0.5 * _randn(g, e)
        w, ids = torch.topk(torch.softmax(logits, -1), case["top_k"], dim=-1)
        s["ids"], s["weights"] = ids.to(torch.int32), w / w.sum(-1, keepdim=True)
        s["gate"], s["up"] = _weights(g, e * inner, K), _weights(g, e * inner, K)
        s["down"] = _weights(g, e * K, inner)
        s["b_inner"] = _pow2(g, e * inner, -1, 1)
        s["residual"] = _stream(g, tokens, K).to(dt) if case["residual"] else None
        return s
    out, n, r = case["out"], case["adapters"], case["rank"]
    X = _stream(g, tokens, K).to(torch.bfloat16)
    s["X"] = X
    s["b"] = _pow2(g, K, -1, 1)  # the weights' column inverse scales: the product reads X D_b
    s["codes"], s["scales"] = _activations(X.float() * s["b"], case["act_fmt"])
    s["w"] = _weights(g, out, K)
    s["adapter"] = _requests(g, case)
    s["A"] = (_randn(g, n, r, K) * (1.0 / math.sqrt(K))).to(torch.bfloat16)
    s["B"] = (_randn(g, n, out, r) * (0.5 / math.sqrt(r))).to(torch.bfloat16)
    s["scale"] = 0.5 + torch.rand(n, device="cuda", generator=g)
    s["bias"] = _randn(g, out) if case["bias"] else None
    s["residual"] = _randn(g, tokens, out).to(dt) if case["residual"] else None
    return s


# ------------------------------------------------------------------------- the plain form


def _quantize_values(x, fmt):
    """Group quantization of fp32 rows: the exponents e of the E8M0 scales (floor(log2 max) less
    the element type's largest exponent, in [-126, 126]; 0 for a group of zeros) and the
    element values v (x ~ v * 2^e)."""
    rows, cols = x.shape
    mx = x.abs().view(rows, cols // GROUP, GROUP).amax(-1)
    emax, top = (2, 6.0) if fmt == "mxfp4" else (8, 448.0)
    e = torch.frexp(mx).exponent - 1 - emax
    e = torch.where(mx > 0, e.clamp(-126, 126), torch.zeros_like(e))
    v = x.view(rows, cols // GROUP, GROUP) * torch.exp2(-e.float())[..., None]
    v = v.clamp(-top, top).view(rows, cols)
    if fmt == "mxfp4":
        m = v.abs()
        step = torch.where(m < 2.0, 0.5, torch.where(m < 4.0, 1.0, 2.0))
        v = torch.round(v / step) * step
    else:
        v = v.to(torch.float8_e4m3fn).float()
    return e, v


def _fp4_codes(v):
    m = v.abs()
    idx = torch.where(m < 2.0, 2.0 * m, torch.where(m < 4.0, m + 2.0, 0.5 * m + 4.0))
    code = idx.to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _fp8_codes(v):
    return torch.where(v == 0, torch.zeros_like(v), v).to(torch.float8_e4m3fn).view(torch.uint8)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _decode(codes, scales, fmt):
    """rows x K fp32 values of codes and E8M0 bytes."""
    if fmt == "mxfp4":
        pairs = torch.tensor([(a, b) for b in _E2M1 for a in _E2M1], device=codes.device)
        v = pairs[codes.int()].flatten(1)
    else:
        v = codes.view(torch.float8_e4m3fn).float()
    d = torch.exp2(scales.float() - 127.0)
    return (v.view(v.shape[0], -1, GROUP) * d[..., None]).view(v.shape)


def _act(z, kind):
    if kind == "none":
        return z
    if kind == "relu":
        return z.clamp_min(0.0)
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _rstd(x):
    return (1.0 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + EPS)).float()


def _plain_norm(s):
    # one fp32 rounding per step, the means of squares in float64: x is next to the borders of
    # the quantizer
    m = s["X"].float()
    if s["post"] is not None:
        m = m * _rstd(m) * s["post"].float()
    if s["gate"] is not None:
        m = m * s["gate"]
    if s["token_gate"] is not None:
        m = m * s["token_gate"][:, None]
    h = (s["residual"].float() * s["residual_scale"] + m).to(s["X"].dtype)
    n = h.float() * _rstd(h.float()) * s["weight"].float()
    e, v = _quantize_values(n * s["b"], "mxfp8")
    out = dict(residual=h, codes=_fp8_codes(v).view(torch.float8_e4m3fn),
               scales=(e + 127).to(torch.uint8).view(torch.float8_e8m0fnu))
    return dict(out, x=n.to(s["X"].dtype)) if s["case"]["x_out"] else out


def _plain_route(s):
    c = s["case"]
    logits = torch.matmul(s["X"].double(), s["W"].double().t()).float().double()
    p = torch.softmax(logits, -1) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-logits))
    key = p if s["bias"] is None else p + s["bias"].double()
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = torch.gather(p, 1, ids)
    return dict(ids=ids.to(torch.int32), weights=(w / w.sum(-1, keepdim=True)).float())


def _rows(w, ids, experts):
    """Weights (experts x rows x K) and row scales of the experts in ids, or of all."""
    codes = w["codes"].view(experts, -1, w["codes"].shape[1])
    scales, a = w["scales"].view(experts, -1, w["scales"].shape[1]), w["a"].view(experts, -1)
    if ids is not None:
        codes, scales, a = codes[ids], scales[ids], a[ids]
    v = _decode(codes.flatten(0, 1), scales.flatten(0, 1), "mxfp4")
    return v.view(codes.shape[0], codes.shape[1], -1), a


def _plain_moe(s):
    c = s["case"]
    t, k, n, inner = c["tokens"], c["top_k"], c["experts"], c["inner"]
    x = _decode(s["codes"], s["scales"], c["act_fmt"])
    ids = s["ids"].long()
    few = t * k <= n  # gather the pairs' experts, or compute every expert for every token
    # experts (or pairs) x tokens x channels
    x = x.repeat_interleave(k, dim=0)[:, None] if few else x[None].expand(n, -1, -1)
    of = ids.flatten() if few else None

    def product(v, w):
        q, a = _rows(w, of, n)
        return torch.matmul(v, q.transpose(1, 2)) * a[:, None]

    h = _act(product(x, s["gate"]), c["act"]) * product(x, s["up"])
    b = s["b_inner"].view(n, 1, inner)
    e, v = _quantize_values((h * (b[of] if few else b)).flatten(0, 1), "mxfp8")
    v = (v.view(*e.shape, GROUP) * torch.exp2(e.float())[..., None]).view(h.shape)
    y = product(v, s["down"])
    if few:
        y = y.view(t, k, -1)
    else:
        y = y[ids, torch.arange(t, device=ids.device)[:, None]]
    y = (y * s["weights"][..., None]).sum(1)
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return y.to(torch.bfloat16)


def _plain_adapter(s):
    c = s["case"]
    n, r = c["adapters"], c["rank"]
    x = _decode(s["codes"], s["scales"], c["act_fmt"])
    z = (x @ _decode(s["w"]["codes"], s["w"]["scales"], "mxfp4").t()) * s["w"]["a"]
    if s["bias"] is not None:
        z = z + s["bias"]
    u = torch.matmul(s["X"].float(), s["A"].float().flatten(0, 1).t()).view(-1, n, r)
    mine = s["adapter"][:, None] == torch.arange(n, device=u.device)[None]
    u = torch.where(mine[..., None], u * s["scale"][:, None], torch.zeros_like(u))
    z = z + torch.matmul(u.flatten(1), s["B"].float().transpose(1, 2).flatten(0, 1))
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return y.to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)


# ---------------------------------------------------------------- the framework's kernels


def _own_norm(dq, s):
    X = s["X"]
    codes, scales = dq.act_outputs(X, "mxfp8", GROUP)
    h = torch.empty_like(X)
    x = torch.empty_like(X) if s["case"]["x_out"] else None
    dq.block_norm_quantize_act_async(X, "mxfp8", GROUP, codes, scales, s["status"],
                                     residual=s["residual"], residual_out=h, x_out=x,
                                     post_norm=s["post"] is not None, post_weight=s["post"],
                                     gate=s["gate"], token_gate=s["token_gate"],
                                     residual_scale=s["residual_scale"], weight=s["weight"],
                                     b=s["b"], post_eps=EPS, eps=EPS)
    out = dict(residual=h, codes=codes.view(torch.float8_e4m3fn),
               scales=scales.view(torch.float8_e8m0fnu))
    return out if x is None else dict(out, x=x)


def _own_route(dq, s):
    c = s["case"]
    ids, weights = dq.moe_route(s["X"], s["W"], c["top_k"], score=c["score"], bias=s["bias"],
                                renormalize=True)
    return dict(ids=ids, weights=weights)


def _own_moe(dq, s):
    c = s["case"]
    return dq.moe_mx(s["codes"], s["scales"], s["ids"], s["weights"], s["gate"]["packed"],
                     s["up"]["packed"], s["down"]["packed"], c["experts"], a_gate=s["gate"]["a"],
                     a_up=s["up"]["a"], a_down=s["down"]["a"], activation=c["act"],
                     b_inner=s["b_inner"], residual=s["residual"], act_fmt=c["act_fmt"],
                     inner_fmt="mxfp8")


def _own_adapter(dq, s):
    c = s["case"]
    return dq.gemm_mx_adapters(s["codes"], s["scales"], s["w"]["packed"], s["X"], s["adapter"],
                               s["A"], s["B"], scale=s["scale"], a=s["w"]["a"], bias=s["bias"],
                               activation=c["act"], residual=s["residual"], act_fmt=c["act_fmt"],
                               out_dtype=c["dtype"])


def run(state):
    op = state["case"]["op"]
    if own:
        import dual_scale_w4a4_amd as dq

        return dict(norm=_own_norm, route=_own_route, moe=_own_moe, adapter=_own_adapter)[op](
            dq, state)
    return dict(norm=_plain_norm, route=_plain_route, moe=_plain_moe, adapter=_plain_adapter)[op](
        state)


# ------------------------------------------------------------------------------ the work


def work(case):
    op, t = case["op"], case["tokens"]
    q = lambda n, fmt: n * (0.5 if fmt == "mxfp4" else 1.0) + n / GROUP  # noqa: E731
    es = 4 if case.get("dtype") == "f32" else 2
    if op == "norm":
        n = case["cols"]
        streams = 4 if case["x_out"] else 3
        return dict(bytes=t * n * es * streams + n * (es * (2 if case["post"] else 1) + 4 +
                                                      (4 if case["gate"] else 0)) +
                    (4 * t if case["token_gate"] else 0) + q(t * n, "mxfp8"), flops=14.0 * t * n)
    if op == "route":
        n, e, k = case["cols"], case["experts"], case["top_k"]
        return dict(bytes=es * n * (t + e) + 8 * t * k + (4 * e if case["bias"] else 0),
                    flops=2.0 * t * e * n)
    K = case["K"]
    w = lambda out, k: q(out * k, "mxfp4") + 4 * out  # noqa: E731
    if op == "moe":
        inner, n, k = case["inner"], case["experts"], case["top_k"]
        active = n * (1.0 - (1.0 - k / n) ** t)  # experts that some token takes, on average
        return dict(bytes=active * (2 * w(inner, K) + 4 * inner + w(K, inner)) +
                    q(t * K, case["act_fmt"]) + 8 * t * k +
                    t * K * 2 * (2 if case["residual"] else 1), flops=6.0 * t * k * K * inner)
    out, r, n = case["out"], case["rank"], case["adapters"]
    used = n * (1.0 - (1.0 - 1.0 / (n + 1)) ** (n + 1 if case["packed"] else t))
    return dict(bytes=q(t * K, case["act_fmt"]) + w(out, K) + 2 * t * K + 4 * t +
                used * (2 * r * (K + out) + 4) + t * out * es * (2 if case["residual"] else 1) +
                (4 * out if case["bias"] else 0), flops=2.0 * t * (K * out + r * (K + out)))


# -------------------------------------------------------------- the definitions in 64 bits


def _exact_values(codes, scales, fmt):
    sc = scales.double() - 127.0
    if fmt == "mxfp4":
        nib = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
        mag, sign = nib & 7, 1.0 - 2.0 * (nib >> 3).double()
        # magnitude index m: exponent m >> 1, mantissa bit m & 1
        ex, man = (mag >> 1).double(), (mag & 1).double()
        v = torch.where(ex > 0, (1.0 + 0.5 * man) * torch.exp2(ex - 1.0), 0.5 * man) * sign
    else:
        u = codes.long()
        ex, man = ((u >> 3) & 15).double(), (u & 7).double()
        v = torch.where(ex > 0, (1.0 + man / 8.0) * torch.exp2(ex - 7.0), man * 2.0 ** -9)
        v = v * (1.0 - 2.0 * (u >> 7).double())
    return v * torch.exp2(sc).repeat_interleave(GROUP, dim=1)


def _exact_quantize8(x):
    """Element values and scale values of the MXFP8 quantizer in float64."""
    mx = x.abs().unflatten(1, (-1, GROUP)).amax(-1)
    lg = torch.floor(torch.log2(mx.clamp_min(2.0 ** -1000)))
    lg = torch.where(torch.exp2(lg + 1.0) <= mx, lg + 1.0, lg)  # log2 rounds at powers of two
    lg = torch.where(torch.exp2(lg) > mx, lg - 1.0, lg)
    d = torch.exp2(torch.where(mx > 0, (lg - 8).clamp(-126, 126), torch.zeros_like(lg)))
    u = (x / d.repeat_interleave(GROUP, dim=1)).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -100))).clamp_min(-6) - 3)
    return torch.round(u / step) * step, d


def _exact_act(z, kind):
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return torch.relu(z) if kind == "relu" else z


def _exact_norm(s):
    m = s["X"].double()
    if s["post"] is not None:
        m = m * torch.rsqrt((m * m).mean(-1, keepdim=True) + EPS) * s["post"].double()
    for f in (s["gate"], None if s["token_gate"] is None else s["token_gate"][:, None]):
        m = m if f is None else m * f.double()
    h = (s["residual"].double() * s["residual_scale"] + m).to(s["X"].dtype).double()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].double()
    v, d = _exact_quantize8(n * s["b"].double())
    out = dict(residual=h, codes=v, scales=d)
    return dict(out, x=n) if s["case"]["x_out"] else out


def _exact_route(s):
    c = s["case"]
    z = (s["X"].double() @ s["W"].double().t()).to(torch.float32).double()
    if c["score"] == "softmax":
        p = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
    else:
        p = torch.sigmoid(z)
    key = p if s["bias"] is None else p + s["bias"].double()
    order = torch.argsort(-key, dim=-1, stable=True)[:, :c["top_k"]]
    w = torch.take_along_dim(p, order, 1)
    return dict(ids=None, weights=w / w.sum(-1, keepdim=True))


def _exact_moe(s):
    c = s["case"]
    n, inner, K = c["experts"], c["inner"], c["K"]
    x = _exact_values(s["codes"], s["scales"], c["act_fmt"])
    y = torch.zeros(c["tokens"], K, dtype=torch.float64, device="cuda")
    for e in torch.unique(s["ids"]).tolist():
        at, slot = torch.nonzero(s["ids"] == e, as_tuple=True)

        def product(v, w, rows):
            r = slice(e * rows, (e + 1) * rows)
            return (v @ _exact_values(w["codes"][r], w["scales"][r], "mxfp4").t()) * w["a"][r].double()

        h = _exact_act(product(x[at], s["gate"], inner), c["act"]) * product(x[at], s["up"], inner)
        v, d = _exact_quantize8(h * s["b_inner"][e * inner:(e + 1) * inner].double())
        m = product(v * d.repeat_interleave(GROUP, dim=1), s["down"], K)
        y.index_add_(0, at, m * s["weights"][at, slot].double()[:, None])
    return y if s["residual"] is None else s["residual"].double() + y


def _exact_adapter(s):
    c = s["case"]
    x = _exact_values(s["codes"], s["scales"], c["act_fmt"])
    z = (x @ _exact_values(s["w"]["codes"], s["w"]["scales"], "mxfp4").t()) * s["w"]["a"].double()
    if s["bias"] is not None:
        z = z + s["bias"].double()
    for r in torch.unique(s["adapter"][s["adapter"] >= 0]).tolist():
        at = torch.nonzero(s["adapter"] == r).flatten()
        u = (s["X"][at].double() @ s["A"][r].double().t()) * s["scale"][r].double()
        z[at] += u @ s["B"][r].double().t()
    y = _exact_act(z, c["act"])
    return y if s["residual"] is None else s["residual"].double() + y


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, route=_exact_route, moe=_exact_moe, adapter=_exact_adapter)[
        case["op"]](s)
