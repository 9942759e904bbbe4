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
