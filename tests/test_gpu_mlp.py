"""The MLP operators on the GPU against plain float64 implementations (mlp_ref.py).

Norm and quantizer are compared bit for bit with the definition's fp32 steps; products within
the bound their arithmetic gives (mlp_ref.product, act_error), plus half a step of the output
type; quantized products by the quantizer's rule within that bound, and bit for bit where every
sum is exact."""
import numpy as np
import pytest

import mlp_ref as ref
import workloads
from parity import host, scales_np, to_device

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


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


def _bits(x):
    """float32 values that are bf16, as their 16 bits"""
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


# ---------------------------------------------------------------------------------- norm


def _norm_case(tokens, cols, dtype, seed, residual=True, wdt="f32"):
    X = workloads.activations(tokens, cols, seed=seed, dtype=dtype)
    R = workloads.activations(tokens, cols, seed=seed + 1, dtype=dtype) if residual else None
    f32 = workloads.bf16_bits_to_fp32 if dtype == "bf16" else (lambda v: v)
    rng = np.random.default_rng(seed)
    w = (1 + 0.3 * rng.standard_normal(cols)).astype(np.float32)
    if wdt == "bf16":
        w = ref.bf16(w)
    b = np.ldexp(np.float32(1), rng.integers(-3, 4, cols)).astype(np.float32)
    return dict(X=X, R=R, Xf=f32(X), Rf=None if R is None else f32(R), w=w, b=b, wdt=wdt,
                dtype=dtype)


def _norm_want(oracle, c, fmt, group, eps, g=0.0, w=True, b=True):
    h, x = ref.norm(c["Xf"], c["Rf"], c["w"] if w else None, c["b"] if b else None, eps,
                    c["dtype"] == "bf16")
    if fmt == "mxfp8":
        codes, scales = ref.mxfp8(x, group)
    else:
        q = oracle.quantize_act(x, "f32", fmt, group, None, g)
        codes, scales = q["codes"], q["scales"]
    return h, codes, scales


def _norm_check(dq, oracle, c, fmt, group, eps=1e-5, g=0.0, w=True, b=True, inplace=False):
    import torch

    tokens, cols = c["Xf"].shape
    print(f"[norm] {tokens}x{cols} {c['dtype']} {fmt} G={group} R={c['R'] is not None} w={w} "
          f"b={b} inplace={inplace}", flush=True)
    wd = None
    if w:
        wd = to_device(_bits(c["w"]), "bf16") if c["wdt"] == "bf16" else _dev(c["w"])
    R = None if c["R"] is None else to_device(c["R"], c["dtype"])
    got = dq.norm_quantize_act(to_device(c["X"], c["dtype"]), fmt, group, weight=wd, residual=R,
                               residual_out=R if inplace else None, b=_dev(c["b"]) if b else None,
                               eps=eps, g=g)
    torch.cuda.synchronize()
    h, codes, scales = _norm_want(oracle, c, fmt, group, eps, g, w, b)
    if R is not None:
        assert np.array_equal(got["residual"].float().cpu().numpy(), h)
        if inplace:
            assert got["residual"] is R
    bad = np.argwhere(host(got["codes"]) != codes)
    assert bad.size == 0, (len(bad), bad[:4])
    assert np.array_equal(scales_np(got["scales"], fmt), scales)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "mxint4", "nvfp4", "int4_bf16"])
@pytest.mark.parametrize("group", [16, 32, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_every_format(dq, oracle_lib, fmt, group, dtype):
    c = _norm_case(19, 1088, dtype, seed=group, wdt=dtype)
    _norm_check(dq, oracle_lib, c, fmt, group, g=0.004 if fmt == "nvfp4" else 0.0)


@pytest.mark.parametrize("tokens,cols", [(1, 32), (1, 64), (3, 96), (5, 1024), (2, 1056),
                                         (7, 4096), (3, 4128), (2, 8192), (2, 8160), (3, 14336),
                                         (2, 16416), (1, 40960), (130, 4096), (1, 131072)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_shapes(dq, oracle_lib, tokens, cols, dtype):
    c = _norm_case(tokens, cols, dtype, seed=cols + tokens, residual=tokens != 3)
    _norm_check(dq, oracle_lib, c, "mxfp8", 32, inplace=tokens == 2)
    _norm_check(dq, oracle_lib, c, "mxfp4", 32)


@pytest.mark.parametrize("w", [False, True])
@pytest.mark.parametrize("b", [False, True])
@pytest.mark.parametrize("wdt", ["f32", "bf16"])
def test_norm_optional_vectors(dq, oracle_lib, w, b, wdt):
    for dtype in ("bf16", "f32"):
        c = _norm_case(6, 544, dtype, seed=3, wdt=wdt)
        _norm_check(dq, oracle_lib, c, "mxfp8", 32, w=w, b=b, eps=1e-6)


def test_norm_zero_and_tiny_rows(dq, oracle_lib):
    # rows of zeros (also zeros that a residual cancels), of the smallest subnormals, of large
    # values, and groups of zeros between others
    cols = 1024
    X = np.zeros((6, cols), np.float32)
    R = np.zeros((6, cols), np.float32)
    rng = np.random.default_rng(5)
    X[1] = rng.standard_normal(cols)
    R[1] = -X[1]
    X[2] = 2.0 ** -149
    X[3] = 1e30 * rng.standard_normal(cols)
    X[4, 100:130] = rng.standard_normal(30)
    X[5, ::3] = -1e-42
    c = dict(X=X, R=R, Xf=X, Rf=R, w=np.ones(cols, np.float32), b=np.ones(cols, np.float32),
             wdt="f32", dtype="f32")
    for fmt in ("mxfp8", "mxfp4", "mxint4", "int4_bf16"):
        _norm_check(dq, oracle_lib, c, fmt, 32)
    # a weight that carries x far down and far up
    c["w"] = np.where(np.arange(cols) % 64 < 32, np.float32(2.0 ** -100), np.float32(2.0 ** 60))
    for fmt in ("mxfp8", "mxfp4"):
        _norm_check(dq, oracle_lib, c, fmt, 32, eps=1e-30)


def test_norm_ties_of_the_eight_bit_format(dq, oracle_lib):
    # x made of E4M3 midpoints and their neighbours: a row of constant mean square 1 - eps is not
    # at hand, so the weight places the values (x = h r w with r found from the row first)
    cols = 256
    vals = ref.e4m3_values()
    pos = np.unique(vals[np.isfinite(vals) & (vals >= 0)])
    mids = ((pos[:-1] + pos[1:]) / 2).astype(np.float32)
    w = np.resize(np.concatenate([mids, np.nextafter(mids, np.float32(0)),
                                  np.nextafter(mids, np.float32(1e9)), -mids]), cols)
    X = np.ones((4, cols), np.float32)
    X[1] *= -1
    X[2] *= 2
    X[3] *= 0.5
    w[::32] = 448.0  # the scale of every group is 2^0 times the row's r
    eps = 2.0 ** -60
    c = dict(X=X, R=None, Xf=X, Rf=None, w=w.astype(np.float32), b=None, wdt="f32", dtype="f32")
    _norm_check(dq, oracle_lib, c, "mxfp8", 32, eps=eps, b=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_reports_bad_values(dq, oracle_lib, dtype):
    import torch

    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    X = torch.randn(5, 288, device="cuda").to(dt)
    R = torch.randn(5, 288, device="cuda").to(dt)

    def run(X, R, w=None):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        codes, scales = dq.act_outputs(X, "mxfp8", 32)
        h = None if R is None else torch.empty_like(X)
        dq.norm_quantize_act_async(X, "mxfp8", 32, codes, scales, status, weight=w, residual=R,
                                   residual_out=h)
        return int(status.item()), codes, scales

    good = run(X, R)
    assert good[0] == 0
    for v in (float("nan"), float("inf"), float("-inf")):
        for into in ("X", "R"):
            X2, R2 = X.clone(), R.clone()
            (X2 if into == "X" else R2)[2, 133] = v
            st, codes, scales = run(X2, R2)
            assert st == 1, (v, into, st)
            rows = [0, 1, 3, 4]  # other rows are as they were
            assert torch.equal(codes[rows], good[1][rows])
            assert torch.equal(scales[rows], good[2][rows])
            with pytest.raises(dq.DQError) as e:
                dq.norm_quantize_act(X2, "mxfp8", 32, residual=R2)
            assert e.value.status == 3
    big = torch.full_like(X, 3.2e38)
    assert run(big, big)[0] == 2          # the sum overflows
    w = torch.full((288,), 3e38, device="cuda")
    spike = torch.zeros_like(X)
    spike[:, 7] = 1.0                     # x = sqrt(288) * 3e38 overflows in one channel
    assert run(spike, None, w)[0] == 2
    with pytest.raises(dq.DQError) as e:
        dq.norm_quantize_act(spike, "mxfp8", 32, weight=w)
    assert e.value.status == 4


# ------------------------------------------------------------------------------ products


def _acts(tokens, K, fmt, seed, lo=120, hi=135):
    if fmt == "mxfp4":
        return workloads.mx_operands(tokens, K, seed=seed, lo=lo, hi=hi)
    return ref.mxfp8_operand(np.random.default_rng(seed), tokens, K)


def _weights(out, K, seed, lo=118, hi=124):
    wc, ws = workloads.mx_operands(out, K, seed=seed, lo=lo, hi=hi)
    a = np.random.default_rng(seed).uniform(0.1, 1.5, out).astype(np.float32)
    a /= np.float32(np.sqrt(K))
    return wc, ws, a


def _pack(dq, wc, ws):
    return dq.gemm_pack_weights(_dev(wc), _dev(ws))


def _residual(rng, tokens, out, dtype):
    r = rng.standard_normal((tokens, out)).astype(np.float32)
    if dtype == "f32":
        return r, _dev(r)
    r = ref.bf16(r)
    return r, to_device(_bits(r), "bf16")


def _sampled(rng, n, sample):
    """All of 0 .. n - 1, or about `sample` of them: both ends, the neighbours of every 256-tile
    edge and others at random."""
    if sample is None or n <= sample:
        return np.arange(n)
    edges = np.concatenate([np.arange(0, n, 256), np.arange(255, n, 256), [0, n - 1]])
    rest = rng.choice(n, max(1, sample - len(edges)), replace=False)
    return np.unique(np.concatenate([edges, rest]))


def _epilogue_check(dq, tokens, out, K, act_fmt="mxfp4", dtype="bf16", kind="none", a=True,
                    bias=False, residual=False, inplace=False, seed=0, sample=None):
    print(f"[epilogue] tokens={tokens} out={out} K={K} {act_fmt}->{dtype} {kind} a={a} bias={bias} "
          f"res={residual} inplace={inplace}", flush=True)
    rng = np.random.default_rng(seed + 77)
    xc, xs = _acts(tokens, K, act_fmt, seed + 1)
    wc, ws, av = _weights(out, K, seed + 2)
    av = av if a else None
    bv = rng.standard_normal(out).astype(np.float32) if bias else None
    rh, rd = _residual(rng, tokens, out, dtype) if residual else (None, None)
    y = dq.gemm_mx_epilogue(_dev(xc), _dev(xs), _pack(dq, wc, ws), a=_dev(av), bias=_dev(bv),
                            activation=kind, residual=rd, act_fmt=act_fmt, out_dtype=dtype,
                            y=rd if inplace else None)
    ts, cs = _sampled(rng, tokens, sample), _sampled(rng, out, sample)
    want, dy = ref.epilogue(xc[ts], xs[ts], act_fmt, wc[cs], ws[cs], None if av is None else av[cs],
                            None if bv is None else bv[cs], kind,
                            None if rh is None else rh[np.ix_(ts, cs)])
    ref.check_rounded(_f64(y)[np.ix_(ts, cs)], want, dy, dtype)


# tokens, channels, K: single tokens, ragged sizes, every k count around the waves' shares, and
# sizes that reach each kernel of the selection (32 x 32 blocks: up to 256, 512, 1024 and beyond;
# tiles of 64 tokens up to 256 of them, then of 128)
SHAPES = [(1, 4, 512), (1, 70, 1024), (2, 1000, 512), (17, 33, 1536), (32, 256, 512),
          (33, 260, 2048), (64, 96, 5120), (97, 131, 1024), (128, 512, 512), (130, 300, 2560),
          (256, 256, 1024), (300, 520, 1536), (20, 9000, 512), (31, 8212, 1536),
          (160, 3200, 1024), (300, 3300, 512), (333, 4004, 1536), (510, 6000, 512),
          (700, 9001, 512), (1030, 5555, 1024)]


@pytest.mark.parametrize("tokens,out,K", SHAPES)
@pytest.mark.parametrize("act_fmt,dtype", [("mxfp4", "bf16"), ("mxfp4", "f32"), ("mxfp8", "bf16")])
def test_epilogue_shapes(dq, tokens, out, K, act_fmt, dtype):
    _epilogue_check(dq, tokens, out, K, act_fmt, dtype, residual=True, seed=tokens, sample=300)


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("act_fmt,dtype", [("mxfp4", "bf16"), ("mxfp4", "f32"), ("mxfp8", "bf16")])
@pytest.mark.parametrize("tokens,out", [(5, 100), (140, 264)])
def test_epilogue_activations(dq, kind, act_fmt, dtype, tokens, out):
    for a, bias, residual, inplace in ((True, True, False, False), (False, False, True, True),
                                       (True, True, True, True)):
        _epilogue_check(dq, tokens, out, 512, act_fmt, dtype, kind, a, bias, residual, inplace,
                        seed=11)


@pytest.mark.parametrize("tokens", [3, 200])
def test_epilogue_unaligned_output(dq, tokens):
    # Y and residual aligned to their element only, inside a larger array whose other values stay
    import torch

    out, K = 64, 512
    xc, xs = _acts(tokens, K, "mxfp4", 3)
    wc, ws, a = _weights(out, K, 4)
    for dtype, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        rng = np.random.default_rng(5)
        rh, rd = _residual(rng, tokens, out, dtype)
        big = torch.full((tokens * out + 8,), 7.0, dtype=dt, device="cuda")
        y = big[1:1 + tokens * out].view(tokens, out)
        dq.gemm_mx_epilogue(_dev(xc), _dev(xs), _pack(dq, wc, ws), a=_dev(a), residual=rd,
                            out_dtype=dtype, y=y)
        want, dy = ref.epilogue(xc, xs, "mxfp4", wc, ws, a, None, "none", rh)
        ref.check_rounded(_f64(y), want, dy, dtype)
        assert float(big[0]) == 7.0 and torch.all(big[1 + tokens * out:] == 7.0)


@pytest.mark.parametrize("tokens,out", [(300, 4097), (300, 4100), (1100, 4099), (1100, 4098)])
def test_epilogue_unaligned_tiles(dq, tokens, out):
    # the tile kernels on rows that start at any element, updated in place inside a larger array
    # whose other values stay; rows behind the last token and a ragged end of the channels
    import torch

    K = 512
    xc, xs = _acts(tokens, K, "mxfp4", 13)
    wc, ws, a = _weights(out, K, 14)
    pk = _pack(dq, wc, ws)
    rng = np.random.default_rng(15)
    ts, cs = _sampled(rng, tokens, 300), _sampled(rng, out, 300)
    for dtype, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        for lead in (1, 2, 3):
            print(f"[epilogue] tokens={tokens} out={out} {dtype} lead={lead}", flush=True)
            rh, rd = _residual(rng, tokens, out, dtype)
            behind = 40 * out
            big = torch.full((lead + tokens * out + behind,), 7.0, dtype=dt, device="cuda")
            y = big[lead:lead + tokens * out].view(tokens, out)
            y.copy_(rd)
            dq.gemm_mx_epilogue(_dev(xc), _dev(xs), pk, a=_dev(a), activation="relu", residual=y,
                                out_dtype=dtype, y=y)
            want, dy = ref.epilogue(xc[ts], xs[ts], "mxfp4", wc[cs], ws[cs], a[cs], None, "relu",
                                    rh[np.ix_(ts, cs)])
            ref.check_rounded(_f64(y)[np.ix_(ts, cs)], want, dy, dtype)
            assert torch.all(big[:lead] == 7.0) and torch.all(big[lead + tokens * out:] == 7.0)


def test_epilogue_channels_past_two_million(dq):
    # whole tiles whose rows lie further apart than a 31-bit tile offset allows: 4096 weight rows
    # repeated, so that every block of 4096 channels must equal the first, in place on a residual
    import torch

    tokens, K, rows, out = 130, 512, 4096, (1 << 21) + 36
    print(f"[epilogue] tokens={tokens} out={out}", flush=True)
    xc, xs = _acts(tokens, K, "mxfp4", 6)
    wc, ws, _ = _weights(rows, K, 7)
    many = lambda w: _dev(w).repeat(out // rows + 1, 1)[:out].contiguous()  # noqa: E731
    pk = dq.gemm_pack_weights(many(wc), many(ws))
    y = torch.full((tokens, out), 2.0, dtype=torch.bfloat16, device="cuda")
    assert dq.gemm_mx_epilogue(_dev(xc), _dev(xs), pk, residual=y, y=y) is y
    whole = y[:, :out // rows * rows].view(tokens, -1, rows)
    assert torch.equal(whole, whole[:, :1].expand_as(whole))
    assert torch.equal(y[:, out // rows * rows:], y[:, :out % rows])
    ts = _sampled(np.random.default_rng(8), tokens, 16)
    want, dy = ref.epilogue(xc[ts], xs[ts], "mxfp4", wc, ws, None, None, "none",
                            np.full((len(ts), rows), 2.0))
    ref.check_rounded(_f64(y[:, :rows])[ts], want, dy, "bf16")


def _gated_check(dq, tokens, inner, K, act_fmt="mxfp4", dtype="bf16", kind="silu", a=True, seed=0,
                 sample=None):
    print(f"[gated] tokens={tokens} inner={inner} K={K} {act_fmt}->{dtype} {kind} a={a}", flush=True)
    xc, xs = _acts(tokens, K, act_fmt, seed + 1)
    gate, up = _weights(inner, K, seed + 2), _weights(inner, K, seed + 3)
    if not a:
        gate, up = (*gate[:2], None), (*up[:2], None)
    gp, upk = _pack(dq, *gate[:2]), _pack(dq, *up[:2])
    rng = np.random.default_rng(seed + 8)
    ts = _sampled(rng, tokens, sample)
    if dtype in ("bf16", "f32"):
        cs = _sampled(rng, inner, sample)
    else:  # whole groups of 32 channels
        gs = _sampled(rng, inner // 32, None if sample is None else sample // 32)
        cs = (gs[:, None] * 32 + np.arange(32)).reshape(-1)
    cut = lambda w: (w[0][cs], w[1][cs], None if w[2] is None else w[2][cs])  # noqa: E731
    want, dh = ref.gated(xc[ts], xs[ts], act_fmt, cut(gate), cut(up), kind)
    kw = dict(a_gate=_dev(gate[2]), a_up=_dev(up[2]), activation=kind, act_fmt=act_fmt)
    if dtype in ("bf16", "f32"):
        h = dq.gated_mx(_dev(xc), _dev(xs), gp, upk, out_dtype=dtype, **kw)
        ref.check_rounded(_f64(h)[np.ix_(ts, cs)], want, dh, dtype)
        return
    b = np.random.default_rng(seed + 9).uniform(0.5, 2.0, inner).astype(np.float32) if a else None
    q = dq.gated_mx_quantized(_dev(xc), _dev(xs), gp, upk, dtype, b=_dev(b), **kw)
    if b is not None:
        want, dh = want * b[cs], dh * b[cs] + np.abs(want * b[cs]) * ref.U24
    codes = host(q["codes"])
    per = codes.shape[1] * 32 // inner  # code bytes of a group
    codes = codes.reshape(tokens, inner // 32, per)[np.ix_(ts, gs)].reshape(len(ts), -1)
    ref.check_quantized(codes, host(q["scales"])[np.ix_(ts, gs)], want, dh, dtype)


@pytest.mark.parametrize("tokens,inner,K", [(1, 32, 512), (1, 1056, 1024), (2, 64, 512),
                                            (31, 96, 1536), (32, 256, 512), (33, 160, 2048),
                                            (64, 128, 5120), (100, 416, 1024), (129, 256, 512),
                                            (256, 128, 1024), (300, 544, 1536),
                                            (20, 22560, 512), (90, 8000, 512), (190, 5632, 1536),
                                            (400, 3200, 1024), (610, 6464, 512)])
@pytest.mark.parametrize("act_fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp4", "mxfp8"])
def test_gated_shapes(dq, tokens, inner, K, act_fmt, dtype):
    if dtype == "f32" and act_fmt == "mxfp8":
        dtype, kind = "bf16", "relu"  # fp32 is refused for MXFP8 activations
    else:
        kind = "silu"
    _gated_check(dq, tokens, inner, K, act_fmt, dtype, kind, seed=tokens, sample=320)


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp4", "mxfp8"])
def test_gated_activations(dq, kind, dtype):
    for tokens, inner in ((4, 64), (150, 288)):
        _gated_check(dq, tokens, inner, 512, "mxfp4", dtype, kind, seed=21)
        _gated_check(dq, tokens, inner, 512, "mxfp4", dtype, kind, a=False, seed=22)


@pytest.mark.parametrize("tokens,inner", [(1, 37), (40, 1002), (260, 301)])
@pytest.mark.parametrize("act_fmt,dtype", [("mxfp4", "bf16"), ("mxfp4", "f32"), ("mxfp8", "bf16")])
def test_gated_odd_channels(dq, tokens, inner, act_fmt, dtype):
    _gated_check(dq, tokens, inner, 512, act_fmt, dtype, seed=31)


@pytest.mark.parametrize("tokens,inner", [(300, 3201), (333, 3302), (610, 6467)])
@pytest.mark.parametrize("act_fmt,dtype", [("mxfp4", "bf16"), ("mxfp4", "f32"), ("mxfp8", "bf16")])
def test_gated_odd_channels_in_tiles(dq, tokens, inner, act_fmt, dtype):
    _gated_check(dq, tokens, inner, 512, act_fmt, dtype, seed=33, sample=320)


@pytest.mark.parametrize("tokens", [1, 40, 300])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_gated_quantized_is_exact_where_the_sums_are(dq, oracle_lib, tokens, fmt):
    # scales 2^-1 .. 2^1 and power-of-two a, b: sums within 24 bits; relu and the product are then
    # exact or rounded once, so codes and scales are the quantizer's of the exact fp32 values
    K, inner = 512, 320
    xc, xs = _acts(tokens, K, "mxfp4", 41, 126, 129)
    rng = np.random.default_rng(42)
    a = (2.0 ** rng.integers(-3, 4, inner)).astype(np.float32)
    b = (2.0 ** rng.integers(-3, 4, inner)).astype(np.float32)
    gate = (*workloads.mx_operands(inner, K, seed=43, lo=126, hi=129), a)
    up = (*workloads.mx_operands(inner, K, seed=44, lo=126, hi=129), a[::-1].copy())
    print(f"[gated] exact tokens={tokens} {fmt}", flush=True)
    want, _ = ref.gated(xc, xs, "mxfp4", gate, up, "relu")
    x = want.astype(np.float32) * b
    q = dq.gated_mx_quantized(_dev(xc), _dev(xs), _pack(dq, *gate[:2]), _pack(dq, *up[:2]), fmt,
                              a_gate=_dev(gate[2]), a_up=_dev(up[2]), activation="relu", b=_dev(b))
    if fmt == "mxfp8":
        codes, scales = ref.mxfp8(x, 32)
    else:
        o = oracle_lib.quantize_act(x, "f32", "mxfp4", 32, None)
        codes, scales = o["codes"], o["scales"]
    assert np.array_equal(host(q["scales"]), scales)
    assert np.array_equal(host(q["codes"]), codes)


@pytest.mark.parametrize("tokens", [20, 280])
@pytest.mark.parametrize("act_fmt", ["mxfp4", "mxfp8"])
def test_nan_scales_reach_their_outputs_only(dq, tokens, act_fmt):
    K, inner = 1024, 96
    xc, xs = _acts(tokens, K, act_fmt, 51)
    gate, up = _weights(inner, K, 52), _weights(inner, K, 53)
    xs, gs = xs.copy(), gate[1].copy()
    xs[7, 3] = 0xFF   # token 7
    gs[40, 20] = 0xFF  # gate channel 40
    print(f"[gated] nan tokens={tokens} {act_fmt}", flush=True)
    gp, upk = _pack(dq, gate[0], gs), _pack(dq, *up[:2])
    kw = dict(a_gate=_dev(gate[2]), a_up=_dev(up[2]), act_fmt=act_fmt)
    h = _f64(dq.gated_mx(_dev(xc), _dev(xs), gp, upk, **kw))
    nan = np.zeros((tokens, inner), bool)
    nan[7], nan[:, 40] = True, True
    assert np.array_equal(np.isnan(h), nan)
    y = _f64(dq.gemm_mx_epilogue(_dev(xc), _dev(xs), gp, a=kw["a_gate"], act_fmt=act_fmt,
                                 activation="relu"))
    assert np.array_equal(np.isnan(y), nan)  # relu keeps a NaN
    q = dq.gated_mx_quantized(_dev(xc), _dev(xs), gp, upk, "mxfp8", **kw)
    groups = nan.reshape(tokens, 3, 32).any(2)
    assert np.array_equal(host(q["scales"]) == 0xFF, groups)
    assert np.all(host(q["codes"]).reshape(tokens, 3, 32)[groups] == 0)


def test_zero_activations_and_weights(dq):
    # zero rows give 0 (and a residual unchanged), zero groups scale 2^0 and zero codes
    for tokens in (2, 257):
        K, out = 512, 64
        xc, xs = _acts(tokens, K, "mxfp4", 61)
        xc = xc.copy()
        xc[1] = 0x88  # a token of negative zeros
        wc, ws, a = _weights(out, K, 62)
        rh, rd = _residual(np.random.default_rng(63), tokens, out, "bf16")
        pk = _pack(dq, wc, ws)
        y = _f64(dq.gemm_mx_epilogue(_dev(xc), _dev(xs), pk, a=_dev(a), residual=rd))
        assert np.array_equal(y[1], rh[1].astype(np.float64))
        for fmt in ("mxfp4", "mxfp8"):
            q = dq.gated_mx_quantized(_dev(xc), _dev(xs), pk, pk, fmt, a_gate=_dev(a), a_up=_dev(a))
            assert np.all(host(q["codes"])[1] == 0) and np.all(host(q["scales"])[1] == 127)


# ------------------------------------------------------------- together, as they are used


def _block_weights(dq, hidden, inner, seed):
    sols = [_weights(o, k, seed + i) for i, (o, k) in enumerate(((inner, hidden), (inner, hidden),
                                                                 (hidden, inner)))]
    return sols, [_pack(dq, *s[:2]) for s in sols]


@pytest.mark.parametrize("tokens", [1, 7, 150, 520])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_mlp_block(dq, oracle_lib, tokens, fmt):
    # norm -> gated -> down with the residual; every step against its definition on the
    # operands that the step before handed over
    hidden, inner = 1024, 1536
    c = _norm_case(tokens, hidden, "bf16", seed=71)
    sols, pk = _block_weights(dq, hidden, inner, 72)
    b2 = np.ldexp(np.float32(1), np.random.default_rng(73).integers(-1, 2, inner)).astype(np.float32)
    print(f"[block] tokens={tokens} {fmt}", flush=True)
    n = dq.norm_quantize_act(to_device(c["X"], "bf16"), fmt, 32, weight=_dev(c["w"]),
                             residual=to_device(c["R"], "bf16"), b=_dev(c["b"]))
    m = dq.gated_mx_quantized(n["codes"], n["scales"], pk[0], pk[1], fmt, a_gate=_dev(sols[0][2]),
                              a_up=_dev(sols[1][2]), b=_dev(b2), act_fmt=fmt)
    y = dq.gemm_mx_epilogue(m["codes"], m["scales"], pk[2], a=_dev(sols[2][2]),
                            residual=n["residual"], act_fmt=fmt, y=n["residual"].clone())
    h, codes, scales = _norm_want(oracle_lib, c, fmt, 32, 1e-5)
    assert np.array_equal(host(n["codes"]), codes) and np.array_equal(host(n["scales"]), scales)
    assert np.array_equal(_f64(n["residual"]), h.astype(np.float64))
    want, dh = ref.gated(codes, scales, fmt, sols[0], sols[1], "silu")
    want, dh = want * b2, dh * b2 + np.abs(want * b2) * ref.U24
    mc, ms = host(m["codes"]), host(m["scales"])
    ref.check_quantized(mc, ms, want, dh, fmt)
    yw, dy = ref.epilogue(mc, ms, fmt, *sols[2], None, "none", h)
    ref.check_rounded(_f64(y), yw, dy, "bf16")


def test_block_in_a_graph_on_other_streams_and_twice(dq):
    # the three calls captured (the calls allocate nothing), replayed on new inputs between eager
    # work, on a side stream, and repeated: the same bits every time
    import torch

    hidden, inner, tokens = 512, 1024, 37
    sols, pk = _block_weights(dq, hidden, inner, 81)
    av = [_dev(s[2]) for s in sols]
    X = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    R = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers():
        codes, scales = dq.act_outputs(X, "mxfp4", 32)
        mc = torch.empty(tokens, inner // 2, dtype=torch.uint8, device="cuda")
        ms = torch.empty(tokens, inner // 32, dtype=torch.uint8, device="cuda")
        return codes, scales, torch.empty_like(X), mc, ms, torch.empty_like(X)

    def block(buf, stream=None):
        codes, scales, h, mc, ms, y = buf
        dq.norm_quantize_act_async(X, "mxfp4", 32, codes, scales, status, residual=R,
                                   residual_out=h, stream=stream)
        dq.gated_mx_quantized(codes, scales, pk[0], pk[1], "mxfp4", a_gate=av[0], a_up=av[1],
                              codes=mc, scales=ms, stream=stream)
        dq.gemm_mx_epilogue(mc, ms, pk[2], a=av[2], residual=h, y=y, stream=stream)

    eager, graphed, side = buffers(), buffers(), buffers()
    block(eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block(graphed)
    s = torch.cuda.Stream()
    for k in range(4):
        X.copy_(torch.randn(tokens, hidden, device="cuda"))
        block(eager)
        g.replay()
        s.wait_stream(torch.cuda.current_stream())
        block(side, stream=s)
        torch.cuda.synchronize()
        for other in (graphed, side):
            assert all(torch.equal(p, q) for p, q in zip(eager, other)), k
    assert int(status.item()) == 0


def test_a_stream_added_to_itself(dq, oracle_lib):
    # X, residual and residual_out the same array
    for dtype in ("bf16", "f32"):
        for cols in (1024, 16416):
            c = _norm_case(5, cols, dtype, seed=87)
            c["R"], c["Rf"] = c["X"], c["Xf"]
            x = to_device(c["X"], dtype)
            got = dq.norm_quantize_act(x, "mxfp8", 32, residual=x, residual_out=x)
            h, codes, scales = _norm_want(oracle_lib, c, "mxfp8", 32, 1e-5, w=False, b=False)
            assert got["residual"] is x and np.array_equal(x.float().cpu().numpy(), h)
            assert np.array_equal(host(got["codes"]), codes)
            assert np.array_equal(host(got["scales"]), scales)


def test_blocking_norm_from_two_threads(dq):
    # the wait lets other Python threads run, and each call reports its own rows' errors
    import threading

    import torch

    X = torch.randn(64, 1024, device="cuda")
    bad = X.clone()
    bad[3, 5] = float("nan")
    want = dq.norm_quantize_act(X, "mxfp8", 32)["codes"]
    seen = {}

    def work(name, x):
        s = torch.cuda.Stream()
        seen[name] = []
        for _ in range(8):
            try:
                q = dq.norm_quantize_act(x, "mxfp8", 32, stream=s)
                seen[name].append(bool(torch.equal(q["codes"], want)))
            except dq.DQError as e:
                seen[name].append(e.status)

    torch.cuda.synchronize()
    ts = [threading.Thread(target=work, args=a) for a in (("good", X), ("bad", bad))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert seen == {"good": [True] * 8, "bad": [3] * 8}


def test_rows_behind_the_last_token_stay(dq):
    import torch

    tokens, K, out = 45, 512, 96
    xc, xs = _acts(64, K, "mxfp4", 91)
    wc, ws, a = _weights(out, K, 92)
    pk = _pack(dq, wc, ws)
    y = torch.full((64, out), 5.0, device="cuda", dtype=torch.bfloat16)
    dq.gemm_mx_epilogue(_dev(xc)[:tokens], _dev(xs)[:tokens], pk, a=_dev(a), y=y[:tokens])
    assert torch.all(y[tokens:] == 5.0)
    codes = torch.full((64, out), 9, device="cuda", dtype=torch.uint8)
    scales = torch.full((64, out // 32), 9, device="cuda", dtype=torch.uint8)
    dq.gated_mx_quantized(_dev(xc)[:tokens], _dev(xs)[:tokens], pk, pk, "mxfp8",
                          codes=codes[:tokens], scales=scales[:tokens])
    assert torch.all(codes[tokens:] == 9) and torch.all(scales[tokens:] == 9)


def test_rows_behind_the_last_token_stay_in_tiles(dq):
    import torch

    tokens, K, out = 205, 512, 5600
    xc, xs = _acts(320, K, "mxfp4", 93)
    pk = _pack(dq, *_weights(out, K, 94)[:2])
    x, s = _dev(xc)[:tokens], _dev(xs)[:tokens]
    for dt, name in ((torch.bfloat16, "bf16"), (torch.float32, "f32")):
        for f in (lambda y: dq.gemm_mx_epilogue(x, s, pk, y=y, out_dtype=name),
                  lambda y: dq.gated_mx(x, s, pk, pk, y=y, out_dtype=name)):
            y = torch.full((320, out), 5.0, device="cuda", dtype=dt)
            f(y[:tokens])
            assert torch.all(y[tokens:] == 5.0) and not torch.all(y[tokens - 1] == 5.0)
    codes = torch.full((320, out), 9, device="cuda", dtype=torch.uint8)
    scales = torch.full((320, out // 32), 9, device="cuda", dtype=torch.uint8)
    dq.gated_mx_quantized(x, s, pk, pk, "mxfp8", codes=codes[:tokens], scales=scales[:tokens])
    assert torch.all(codes[tokens:] == 9) and torch.all(scales[tokens:] == 9)


def test_a_row_does_not_depend_on_its_batch(dq):
    # the same activations as rows of calls of one size: every row's bits agree
    K, out = 1024, 128
    xc, xs = _acts(1, K, "mxfp4", 95)
    wc, ws, a = _weights(out, K, 96)
    pk = _pack(dq, wc, ws)
    for tokens in (5, 64, 300):
        y = _f64(dq.gemm_mx_epilogue(_dev(np.repeat(xc, tokens, 0)), _dev(np.repeat(xs, tokens, 0)),
                                     pk, a=_dev(a), out_dtype="f32"))
        assert np.all(y == y[0])


def test_binding_refuses(dq):
    import torch

    K, out, tokens = 512, 64, 3
    xc, xs = (_dev(v) for v in _acts(tokens, K, "mxfp4", 97))
    wc, ws, a = _weights(out, K, 98)
    pk = _pack(dq, wc, ws)
    X = torch.randn(3, 64, device="cuda")
    bad = [lambda: dq.gemm_mx_epilogue(xc, xs, pk, activation="swish"),
           lambda: dq.gemm_mx_epilogue(xc, xs, pk, act_fmt="nvfp4"),
           lambda: dq.gemm_mx_epilogue(xc, xs, pk, act_fmt="mxfp8"),
           lambda: dq.gemm_mx_epilogue(xc.cpu(), xs, pk),
           lambda: dq.gemm_mx_epilogue(xc, xs.cpu(), pk),
           lambda: dq.gemm_mx_epilogue(xc[:2], xs, pk),
           lambda: dq.gemm_mx_epilogue(xc, xs, pk, a=torch.ones(out - 1, device="cuda")),
           lambda: dq.gemm_mx_epilogue(xc, xs, pk, out_dtype="f16"),
           lambda: dq.gemm_mx_epilogue(xc, xs, pk, residual=torch.ones(3, out, device="cuda")),
           lambda: dq.gemm_mx_epilogue(xc, xs, pk, bias=torch.ones(out, device="cuda").double()),
           lambda: dq.gated_mx(xc, xs, pk, dict(pk, out=32)),
           lambda: dq.gated_mx_quantized(xc, xs, pk, pk, "nvfp4"),
           lambda: dq.norm_quantize_act(X, "fp8", 32),
           lambda: dq.norm_quantize_act(X, "mxfp8", 48),
           lambda: dq.norm_quantize_act(X.t(), "mxfp8", 32),
           lambda: dq.norm_quantize_act(X, "mxfp8", 32, weight=torch.ones(32, device="cuda")),
           lambda: dq.norm_quantize_act(X, "mxfp8", 32, weight=torch.ones(64, device="cuda").half()),
           lambda: dq.norm_quantize_act(X, "mxfp8", 32, residual=X.bfloat16())]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", k)
    with pytest.raises(dq.DQError):
        dq.norm_quantize_act(X, "mxfp8", 32, residual_out=X)
    with pytest.raises(dq.DQError):
        dq.norm_quantize_act(X, "nvfp4", 32)
