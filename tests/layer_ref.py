"""The operators of include/dq_layer.h in plain numpy: the definitions that tests hold the kernels to.

The block norm follows the definition's fp32 roundings one by one (sums of squares and roots in
float64), so that its results are compared bit for bit; the router's logits are float64 sums
rounded once; products come with a bound on the error that the arithmetic allows."""
from __future__ import annotations

import numpy as np

import mlp_ref as ref

F32 = np.float32


def rounded(x, dtype):
    return ref.bf16(x) if dtype == "bf16" else np.asarray(x, F32)


def _rstd(x, eps):
    ms = np.square(x.astype(np.float64)).sum(1) / x.shape[1]
    return (1.0 / np.sqrt(ms + eps)).astype(F32)[:, None]


def block_norm(X, R, post, gate, tgate, rs, w, b, dtype, post_norm=True, post_eps=1e-5, eps=1e-5):
    """(h, n, x): the stored stream, what x_out holds before its rounding, and the quantizer's
    input, float32 arrays of float32 inputs."""
    m = np.asarray(X, F32)
    if post_norm:
        m = m * _rstd(m, post_eps)
        if post is not None:
            m = m * post.astype(F32)
    if gate is not None:
        m = m * gate.astype(F32)
    if tgate is not None:
        m = m * tgate.astype(F32)[:, None]
    r = np.zeros_like(m) if R is None else np.asarray(R, F32)
    h = rounded(r * F32(rs) + m, dtype)
    n = h * _rstd(h, eps)
    if w is not None:
        n = n * w.astype(F32)
    x = n if b is None else n * b.astype(F32)
    assert m.dtype == h.dtype == n.dtype == x.dtype == F32
    return h, n, x


# ---------------------------------------------------------------------------------- experts


def _grid(v, e, fmt):
    """Values of float64 v quantized with the group exponents e (one per value)."""
    top, bits, emin = (6.0, 1, 0) if fmt == "mxfp4" else (448.0, 3, -6)
    u = np.clip(v / np.exp2(e), -top, top)
    b = np.maximum(np.floor(np.log2(np.maximum(np.abs(u), 2.0 ** -100))), emin)
    step = np.exp2(b - bits)
    return np.rint(u / step) * step * np.exp2(e)


def quantized(x, dx, fmt):
    """(q, dq): the quantizer's values for rows x, and how far those of any values within dx of
    x can be from them: rounding is monotone, so for each scale that a group's largest magnitude
    within reach can give, the ends of each interval are the furthest."""
    emax = 2 if fmt == "mxfp4" else 8
    n = x.shape[0]
    g, d = np.abs(x).reshape(n, -1, 32), dx.reshape(n, -1, 32)
    at = lambda m: np.repeat(ref.mx_exponent(m.max(2), emax), 32, 1).astype(float)  # noqa: E731
    q = _grid(x, at(g), fmt)
    # at most one power of two apart: every test's dx is far below its group's largest value, or
    # the group is all zeros within reach (then every candidate is zero or below dx)
    ends = [_grid(v, at(m), fmt) for v in (x - dx, x + dx) for m in (np.maximum(g - d, 0), g + d)]
    return q, np.max([np.abs(v - q) for v in ends], 0)


def product_whole(xc, xs, act_fmt, wc, ws, a):
    """(z, dz) of ref.product for the experts' first products, where E4M3 activations are multiplied
    in two parts: each part's products are added exactly in runs of 8 but for the last bit of those
    of codes below 4 (2^-10 times both scales at most, 32 to a group); one more matrix step per 64 k."""
    if act_fmt == "mxfp4":
        return ref.product(xc, xs, act_fmt, wc, ws, a)
    x, q = ref.decode(xc, xs, act_fmt), ref.decode(wc, ws, "mxfp4")
    a = np.ones(q.shape[0]) if a is None else np.asarray(a, np.float64)
    scale = lambda s: np.where(s == 255, np.nan, np.exp2(s.astype(float) - 127))  # noqa: E731
    with np.errstate(invalid="ignore"):
        z, S = x @ q.T, np.abs(x) @ np.abs(q).T
        dz = (x.shape[1] / 32 + 2) * 2 * ref.U24 * S + 32 * 2.0 ** -10 * (scale(xs) @ scale(ws).T)
    return z * a, dz * np.abs(a)


def gated_whole(xc, xs, act_fmt, gate, up, kind):
    g, dg = product_whole(xc, xs, act_fmt, *gate)
    u, du = product_whole(xc, xs, act_fmt, *up)
    f, df = ref.act(g, kind), ref.act_error(g, dg, kind)
    return f * u, (np.abs(f) + df) * du + df * np.abs(u) + np.abs(f * u) * ref.U24


def moe(xc, xs, act_fmt, ids, weights, gate, up, down, kind, b, mid, residual):
    """(y, dy) before the rounding to the output type; gate, up, down: (codes, scales, a) with
    experts as a first axis, b experts x inner or None."""
    tokens, out = ids.shape[0], down[0].shape[1]
    y, dy, size = np.zeros((tokens, out)), np.zeros((tokens, out)), np.zeros((tokens, out))
    for e in range(gate[0].shape[0]):
        t, s = np.nonzero(ids == e)
        if not len(t):
            continue
        one = lambda w: (w[0][e], w[1][e], None if w[2] is None else w[2][e])  # noqa: E731
        h, dh = gated_whole(xc[t], xs[t], act_fmt, one(gate), one(up), kind)
        if b is not None:
            h, dh = h * b[e], dh * b[e] + np.abs(h * b[e]) * ref.U24
        q, dq = quantized(h, dh, mid)
        w = ref.decode(down[0][e], down[1][e], "mxfp4")
        K = q.shape[1]
        z, S = q @ w.T, np.abs(q) @ np.abs(w).T
        dz = (K / 64 + 2) * 2 * ref.U24 * S + dq @ np.abs(w).T
        if mid == "mxfp8":  # the matrix instruction aligns 16 products to 2^-13 of the largest
            qa, wa = np.abs(q).reshape(len(q), -1, 16), np.abs(w).reshape(len(w), -1, 16)
            for k in range(K // 16):
                dz += 16 * 2.0 ** -13 * (qa[:, None, k] * wa[None, :, k]).max(-1)
        if down[2] is not None:
            z, dz = z * down[2][e], dz * np.abs(down[2][e])
        v = weights[t, s].astype(np.float64)[:, None]
        np.add.at(y, t, z * v)
        np.add.at(dy, t, dz * np.abs(v))
        np.add.at(size, t, np.abs(z * v))
    dy += size * (ids.shape[1] + 1) * ref.U24
    if residual is not None:
        y = y + residual.astype(np.float64)
        dy += np.abs(y) * ref.U24
    return y, dy


# ---------------------------------------------------------------------------------- router


def logits(X, W):
    return (X.astype(np.float64) @ W.astype(np.float64).T).astype(F32)


def route(l, top_k, score, bias, renormalize, scale):
    """(ids, weights float64) of float32 logits by the definition."""
    l = l.astype(np.float64)
    with np.errstate(all="ignore"):
        if score == "softmax":
            s = np.exp(l - l.max(1, keepdims=True))
            s = s / s.sum(1, keepdims=True)
        else:
            s = 1.0 / (1.0 + np.exp(-l))
        key = s if bias is None else s + bias.astype(np.float64)
    key = np.where(np.isnan(key), -np.inf, key)
    ids = np.argsort(-key, 1, kind="stable")[:, :top_k]
    w = np.take_along_axis(s, ids, 1)
    if renormalize:
        d = w.sum(1, keepdims=True)
        w = np.where(d == 0, 0.0, w / np.where(d == 0, 1.0, d))
    return ids.astype(np.int32), w * scale


# --------------------------------------------------------------------------------- adapters


def adapters(xc, xs, act_fmt, wc, ws, a, bias, kind, res, X, adapter, A, B, scale, dtype):
    """(y, dy) before the rounding to the output type. u is a sum of K exact products in fp32 in
    some order: K roundings of at most 2^-23 of the magnitudes' sum each. Its split into bf16 values
    leaves 2^-18 of it (nearest, twice 9 bits) for bf16 outputs and nothing over 2^-24 for fp32; the
    sum over the rank (three parts at most) rounds like u's."""
    z, dz = ref.product(xc, xs, act_fmt, wc, ws, a)
    for r in range(A.shape[0]):
        t = np.nonzero(adapter == r)[0]
        if not len(t):
            continue
        x, Ar, Br = X[t].astype(np.float64), A[r].astype(np.float64), B[r].astype(np.float64)
        s = 1.0 if scale is None else float(scale[r])
        u, S = x @ Ar.T * s, np.abs(x) @ np.abs(Ar).T * abs(s)
        du = S * (x.shape[1] + 2) * 2.0 ** -23 + np.abs(u) * (2.0 ** -18 if dtype == "bf16" else ref.U24)
        d, D = u @ Br.T, np.abs(u) @ np.abs(Br).T
        z[t] += d
        dz[t] += du @ np.abs(Br).T + D * (3 * Br.shape[1] + 2) * 2.0 ** -23 + np.abs(z[t]) * ref.U24
    if bias is not None:
        z = z + bias.astype(np.float64)
        dz = dz + np.abs(z) * ref.U24
    y, dy = ref.act(z, kind), ref.act_error(z, dz, kind)
    if res is not None:
        y = y + res.astype(np.float64)
        dy = dy + np.abs(y) * ref.U24
    return y, dy
