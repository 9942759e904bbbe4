"""The MLP operators at their largest sizes: calls of several launches, rows that lie megabytes
apart, and long sums."""
import numpy as np
import pytest

import mlp_ref as ref
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dq():
    import torch

    assert torch.cuda.is_available()
    import dual_scale_w4a4_amd

    dual_scale_w4a4_amd.lib()
    yield dual_scale_w4a4_amd
    torch.cuda.empty_cache()


def _dev(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "mxint4", "nvfp4", "int4_bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_more_rows_than_one_launch_takes(dq, fmt, dtype):
    # launches of 2^22 rows: every row is that of the same row in a call of its launch alone
    import torch

    rows, edge, cols = (1 << 22) + 1037, 1 << 22, 32
    print(f"[norm] {rows}x{cols} {dtype} {fmt}", flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(rows, cols, device="cuda", generator=g).to(dt)
    R = torch.randn(rows, cols, device="cuda", generator=g).to(dt)
    kw = dict(group=16 if fmt == "nvfp4" else 32, g=0.01 if fmt == "nvfp4" else 0.0)
    parts = [dq.norm_quantize_act(X[s], fmt, residual=R[s], **kw)
             for s in (slice(0, edge), slice(edge, rows), slice(edge - 5, edge + 7))]
    whole = dq.norm_quantize_act(X, fmt, residual=R, residual_out=R, **kw)
    assert whole["residual"] is R
    for key in ("codes", "scales", "residual"):
        assert torch.equal(whole[key][:edge], parts[0][key]), key
        assert torch.equal(whole[key][edge:], parts[1][key]), key
        assert torch.equal(whole[key][edge - 5:edge + 7], parts[2][key]), key


def _wide_weights(dq, channels, K, seed, period=4096):
    """Packed weights of `period` rows repeated, and those rows' codes and scales."""
    wc, ws = workloads.mx_operands(period, K, seed=seed, lo=118, hi=124)
    many = lambda w: _dev(w).repeat(-(-channels // period), 1)[:channels].contiguous()  # noqa: E731
    return dq.gemm_pack_weights(many(wc), many(ws)), wc, ws


@pytest.mark.parametrize("form", ["bf16", "f32", "mxfp8 to bf16", "gated bf16", "gated mxfp4",
                                  "gated mxfp8"])
def test_products_of_more_tokens_than_one_launch_takes(dq, form):
    # at this width a launch takes 768 tokens; each token's results are those of a call of its
    # launch alone
    import torch

    channels, K, edge, tokens = (1 << 21) + 64, 512, 768, 768 + 130
    print(f"[limits] tokens={tokens} channels={channels} {form}", flush=True)
    act_fmt = "mxfp8" if form.startswith("mxfp8") else "mxfp4"
    rng = np.random.default_rng(4)
    xc, xs = (ref.mxfp8_operand(rng, tokens, K) if act_fmt == "mxfp8" else
              workloads.mx_operands(tokens, K, seed=5, lo=120, hi=135))
    xc, xs = _dev(xc), _dev(xs)
    pk, _, _ = _wide_weights(dq, channels, K, 6)
    g = torch.Generator(device="cuda").manual_seed(7)
    a = torch.rand(channels, device="cuda", generator=g) / 16

    def call(s, **out):
        if form.startswith("gated"):
            kw = dict(a_gate=a, a_up=a, **out)
            if form == "gated bf16":
                return [dq.gated_mx(xc[s], xs[s], pk, pk, **kw)]
            q = dq.gated_mx_quantized(xc[s], xs[s], pk, pk, form.split()[1], **kw)
            return [q["codes"], q["scales"]]
        return [dq.gemm_mx_epilogue(xc[s], xs[s], pk, a=a, act_fmt=act_fmt,
                                    out_dtype="f32" if form == "f32" else "bf16", **out)]

    if form in ("bf16", "f32"):  # in place on a residual
        y = torch.randn(tokens, channels, device="cuda", generator=g)
        y = y if form == "f32" else y.to(torch.bfloat16)
        parts = [call(s, residual=y[s].clone()) for s in (slice(0, edge), slice(edge, tokens))]
        whole = call(slice(0, tokens), residual=y, y=y)
    else:
        parts = [call(s) for s in (slice(0, edge), slice(edge, tokens))]
        whole = call(slice(0, tokens))
    for w, p, q in zip(whole, *parts):
        assert torch.equal(w[:edge], p) and torch.equal(w[edge:], q)


@pytest.mark.parametrize("channels", [1 << 22, (1 << 22) - 27])
@pytest.mark.parametrize("tokens", [20, 130])  # 130: whole tiles, and one of two rows
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_products_of_the_most_channels(dq, channels, tokens, dtype):
    # rows of up to 2^24 bytes, 127 of them in a tile; every block of 4096 channels equals the first
    import torch

    K, period = 512, 4096
    print(f"[limits] tokens={tokens} channels={channels} {dtype}", flush=True)
    xc, xs = workloads.mx_operands(tokens, K, seed=8, lo=120, hi=135)
    pk, wc, ws = _wide_weights(dq, channels, K, 9)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cut = channels // period * period
    ts = np.unique([0, 1, tokens // 2, tokens - 2, tokens - 1])

    def check(y, want, dy):
        whole = y[:, :cut].view(tokens, -1, period)
        assert torch.equal(whole, whole[:, :1].expand_as(whole))
        assert torch.equal(y[:, cut:], y[:, :channels - cut])
        ref.check_rounded(y[:, :period].double().cpu().numpy()[ts], want, dy, dtype)

    y = torch.full((tokens, channels), 2.0, dtype=dt, device="cuda")
    dq.gemm_mx_epilogue(_dev(xc), _dev(xs), pk, residual=y, y=y, out_dtype=dtype)
    check(y, *ref.epilogue(xc[ts], xs[ts], "mxfp4", wc, ws, None, None, "none",
                           np.full((len(ts), period), 2.0)))
    dq.gated_mx(_dev(xc), _dev(xs), pk, pk, activation="relu", y=y, out_dtype=dtype)
    check(y, *ref.gated(xc[ts], xs[ts], "mxfp4", (wc, ws, None), (wc, ws, None), "relu"))


# 4-bit codes of 0, +-0.5 .. +-4: products with each other are whole numbers of quarters up to 16
_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0])


def _exact_operand(g, rows, K, fmt):
    """Codes (scales 2^0) and float64 values of seeded rows of those values, on the GPU."""
    import torch

    k = torch.randint(0, 7, (rows, K), device="cuda", generator=g, dtype=torch.uint8)
    neg = torch.randint(0, 2, (rows, K), device="cuda", generator=g, dtype=torch.uint8)
    neg = torch.where(k == 0, torch.zeros_like(neg), neg)
    v = torch.from_numpy(_VALUES).cuda()[k.int()] * (1.0 - 2.0 * neg.double())
    if fmt == "mxfp4":
        c = k | (neg << 3)
        codes = (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()
    else:
        codes = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda"), v


# K of real layers, odd numbers of 512-k periods, and the largest; channels and tokens that reach
# each kernel of the selection
@pytest.mark.parametrize("tokens,out,K", [(1, 96, 14336), (3, 40, 1 << 22), (33, 40, 1 << 22),
                                          (130, 33, 1 << 22), (70, 300, 28672), (200, 400, 14848),
                                          (190, 4096, 14336), (300, 4099, 9728), (520, 9000, 8192),
                                          (1030, 9000, 5632), (130, 4200, 1 << 17)])
@pytest.mark.parametrize("act_fmt", ["mxfp4", "mxfp8"])
def test_long_sums_are_exact_where_they_can_be(dq, tokens, out, K, act_fmt):
    # values up to 16 in quarters: a sum of K terms of random signs stays below 2^22, where fp32
    # holds quarters; in the 8-bit mode no product is below 2^-6 of the largest
    import torch

    print(f"[limits] tokens={tokens} out={out} K={K} {act_fmt}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(tokens + out)
    xc, xs, x = _exact_operand(g, tokens, K, act_fmt)
    wc, ws, q = _exact_operand(g, out, K, "mxfp4")
    z = x @ q.t()
    assert float(z.abs().max()) < 2.0 ** 20
    pk = dq.gemm_pack_weights(wc, ws)
    dtype, dt = ("f32", torch.float32) if act_fmt == "mxfp4" else ("bf16", torch.bfloat16)
    y = dq.gemm_mx_epilogue(xc, xs, pk, act_fmt=act_fmt, out_dtype=dtype)
    assert torch.equal(y, z.to(torch.float32).to(dt))
    # the gated form: the product of two exact sums is rounded once to fp32
    h = dq.gated_mx(xc, xs, pk, pk, activation="relu", act_fmt=act_fmt, out_dtype=dtype)
    assert torch.equal(h, (z.clamp_min(0.0) * z).to(torch.float32).to(dt))
