"""The MLP operators in plain numpy, with float64 sums: the definitions that tests hold the kernels to.

Norm and quantizer follow the definition's fp32 roundings one by one, so their results are
compared bit for bit; products come with a bound on the error that the arithmetic allows."""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
U24 = 2.0 ** -24
_erf = np.vectorize(math.erf, otypes=[np.float64])


def bf16(x):
    """float32 values rounded to bf16 (nearest, ties to even), as float32; finite input."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return r.astype(np.uint32).view(np.float32)


def e4m3_values():
    """The value of every E4M3 byte (0x7F and 0xFF are NaN)."""
    b = np.arange(256)
    ex, man = (b >> 3) & 15, b & 7
    v = np.where(ex > 0, (1 + man / 8.0) * 2.0 ** (ex - 7.0), man * 2.0 ** -9)
    v = np.where(b & 0x80, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


def e4m3_codes(v):
    """Bytes of the E4M3 values nearest to float64 v (ties to even, saturating; zero is 0x00)."""
    m = np.minimum(np.abs(v), 448.0)
    e = np.floor(np.log2(np.maximum(m, 2.0 ** -100)))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    r = np.rint(m / step) * step  # at most the next power of two, which is a value
    e = np.maximum(np.floor(np.log2(np.maximum(r, 2.0 ** -100))), -6)
    code = np.where(r < 2.0 ** -6, r * 512, (e + 7) * 8 + (r / 2.0 ** e - 1) * 8).astype(np.uint8)
    return np.where((v < 0) & (code > 0), code | 0x80, code).astype(np.uint8)


def mx_exponent(mx, emax):
    """Exponents of the E8M0 scales of groups with largest magnitude mx (float64, exact)."""
    lg = np.frexp(np.where(mx > 0, mx, 1.0))[1] - 1
    return np.where(mx > 0, np.clip(lg - emax, -126, 126), 0)


def mxfp8(x, group):
    """MXFP8 codes and E8M0 bytes of rows x (float32 or float64)."""
    x = np.asarray(x, np.float64)
    e = mx_exponent(np.abs(x).reshape(x.shape[0], -1, group).max(2), 8)
    return e4m3_codes(x / np.exp2(np.repeat(e, group, 1).astype(float))), (e + 127).astype(np.uint8)


def decode(codes, scales, fmt, group=32):
    """rows x K float64 values of MXFP4 or MXFP8 codes and scales (0xFF: NaN)."""
    if fmt == "mxfp4":
        v = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(codes.shape[0], -1)
    else:
        v = e4m3_values()[codes]
    d = np.where(scales == 255, np.nan, np.exp2(scales.astype(float) - 127))
    return v * np.repeat(d, group, 1)


def norm(X, R, w, b, eps, is_bf16):
    """(h, x): the stored stream and the quantizer's input, float32 arrays."""
    h = np.asarray(X, np.float32)
    if R is not None:
        h = (h + np.asarray(R, np.float32)).astype(np.float32)
        if is_bf16:
            h = bf16(h)
    ms = np.square(h.astype(np.float64)).sum(1) / h.shape[1]
    x = h * (1.0 / np.sqrt(ms + eps)).astype(np.float32)[:, None]
    if w is not None:
        x = x * np.asarray(w, np.float32)
    if b is not None:
        x = x * np.asarray(b, np.float32)
    return h, x


def act(z, kind):
    with np.errstate(over="ignore"):
        if kind == "relu":
            return np.maximum(z, 0.0)
        if kind == "silu":
            return z / (1.0 + np.exp(-z))
        if kind == "gelu":
            return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
        if kind == "gelu_tanh":
            return 0.5 * z * (1.0 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_error(z, dz, kind):
    """Bound on the kernel's error in act(z), its z off by at most dz.

    Slopes: at most 1.13 (silu 1.10, both gelu 1.13). Evaluation: silu and the tanh form are z
    times 1 / (1 + 2^s) with s from z in fp32 roundings that leave it off by at most |s| k 2^-24
    (k = 2 for silu: the constant and the product; 8 for the tanh form's polynomial), which
    changes the sigmoid by the relative amount |s| ln 2 k 2^-24; exp2, the sum, the reciprocal
    and the last product add at most 2^-22. erf is off by at most 2^-21 absolutely (4 of its
    ulps), so its form by |z| 2^-22 and two roundings of relative 2^-24. Results below fp32's
    normal range count 2^-126."""
    dz = 1.13 * dz if kind != "none" else dz
    if kind == "silu":
        return dz + np.abs(act(z, kind)) * (2.0 ** -22 + np.abs(z) * 2 * U24) + 2.0 ** -126
    if kind == "gelu_tanh":
        s = 2 * math.sqrt(2 / math.pi) * np.abs(z + 0.044715 * z ** 3)
        return dz + np.abs(act(z, kind)) * (2.0 ** -22 + s * 8 * U24) + 2.0 ** -126
    if kind == "gelu":
        return dz + np.abs(z) * 2.0 ** -21 + 2.0 ** -126
    return dz


def product(xc, xs, act_fmt, wc, ws, a):
    """(z, dz): a_i sum_k x^ Qhat and a bound on the kernel's error in it.

    Every FP4 product is exact; sums go into fp32 accumulators, one 64-k step an instruction,
    and one fp32 rounding by a: (K / 64 + 2) 2 2^-24 of the sum of magnitudes, whatever the
    order. In the 8-bit mode the products of 16 neighbouring k are aligned to 2^-13 of the
    largest first, so each of the 16 is off by at most that."""
    x, q = decode(xc, xs, act_fmt), decode(wc, ws, "mxfp4")
    K = x.shape[1]
    a = np.ones(q.shape[0]) if a is None else np.asarray(a, np.float64)
    with np.errstate(invalid="ignore"):
        z = x @ q.T
        S = np.abs(x) @ np.abs(q).T
        dz = (K / 64 + 2) * 2 * U24 * S
        if act_fmt == "mxfp8":
            xa, qa = np.abs(x).reshape(len(x), -1, 16), np.abs(q).reshape(len(q), -1, 16)
            for k in range(K // 16):
                dz += 16 * 2.0 ** -13 * (xa[:, None, k] * qa[None, :, k]).max(-1)
    return z * a, dz * np.abs(a)


def epilogue(xc, xs, act_fmt, wc, ws, a, bias, kind, res):
    """(y, dy) before the rounding to the output type."""
    z, dz = product(xc, xs, act_fmt, wc, ws, a)
    if bias is not None:
        z = z + bias.astype(np.float64)
        dz = dz + np.abs(z) * U24
    y, dy = act(z, kind), act_error(z, dz, kind)
    if res is not None:
        y = y + res.astype(np.float64)
        dy = dy + np.abs(y) * U24
    return y, dy


def gated(xc, xs, act_fmt, gate, up, kind):
    """(H, dH) with gate, up = (codes, scales, a), before any rounding to an output type."""
    g, dg = product(xc, xs, act_fmt, *gate)
    u, du = product(xc, xs, act_fmt, *up)
    f, df = act(g, kind), act_error(g, dg, kind)
    return f * u, (np.abs(f) + df) * du + df * np.abs(u) + np.abs(f * u) * U24


def check_rounded(got, y, dy, dtype):
    """got (float64) is y rounded to dtype, y off by at most dy."""
    half = {"bf16": 2.0 ** -8, "f32": U24}[dtype]
    tol = dy + half * (np.abs(y) + dy)
    bad = np.argwhere(~(np.abs(got - y) <= tol))
    assert bad.size == 0, (len(bad), bad[:4], got[tuple(bad[0])], y[tuple(bad[0])],
                           tol[tuple(bad[0])])


def check_quantized(codes, scales, x, dx, fmt):
    """codes and scales are the quantizer's for some values within dx of x: every scale is that
    of a largest magnitude within reach, and every element is within half a step of the value
    (which saturates at the largest code)."""
    top, emax, bits, emin = (6.0, 2, 1, 0) if fmt == "mxfp4" else (448.0, 8, 3, -6)
    n = x.shape[0]
    g = np.abs(x).reshape(n, -1, 32)
    d = dx.reshape(n, -1, 32)
    lo = mx_exponent(np.maximum(g - d, 0).max(2), emax) + 127
    hi = mx_exponent((g + d).max(2), emax) + 127
    zero = np.maximum(g - d, 0).max(2) == 0  # a group that may be zero: 2^0, or any below hi
    ok = (scales <= hi) & ((scales >= lo) | zero) | (zero & (scales == 127))
    assert ok.all(), np.argwhere(~ok)[:4]
    v = decode(codes, np.full_like(scales, 127), fmt)
    s = np.repeat(np.exp2(scales.astype(float) - 127), 32, 1)
    u, du = x / s, dx / s
    m = np.minimum(np.abs(u) + du, top)
    half = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(m, 2.0 ** -40))), emin) - bits - 1)
    bad = np.argwhere(~(np.abs(v - np.clip(u, -top, top)) <= half + du))
    assert bad.size == 0, (len(bad), bad[:4], v[tuple(bad[0])], u[tuple(bad[0])])
    assert not np.any(codes == 0x80) if fmt == "mxfp8" else not np.any(
        ((codes & 15) == 8) | ((codes >> 4) == 8)), "a negative zero"


def mxfp8_operand(rng, rows, K, outliers=True):
    """Seeded MXFP8 activations: codes and scales of N(0, 1) rows with a few large channels."""
    x = rng.standard_normal((rows, K))
    if outliers:
        x[:, rng.random(K) < 0.02] *= 20.0
    return mxfp8(x.astype(np.float32), 32)
