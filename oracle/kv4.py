"""Float64 definitions of the 4-bit key/value cache's operators, with error bounds.

Used by the parity tests.  The rules of the bounds are those of ``oracle.decode``
(u = 2^-23), and one rounding to bf16 is off by at most 2^-8 of the value.
"""

from __future__ import annotations

import numpy as np

from . import quant
from .decode import GROUP, U, blocks, magnitudes, weights

BF16 = 2.0**-8


def append(x, fmt, T=None, g=None):
    """(codes [n, heads, D/2], scales [n, heads, D/G]) of x [n, heads, D] (bf16
    values in float64) after the transforms T [heads, D/G, G, G]."""
    n, h, D = x.shape
    y = x if T is None else blocks(x, T[None])[0]
    y = y.astype(np.float32).reshape(n * h, D)
    if fmt == "mxfp4":
        c, s = quant.quant_mxfp4_ref(y)
    elif fmt == "nvfp4":
        c, s = quant.quant_nvfp4_ref(y, g)
    else:
        c, s = quant.quant_int4_ref(y)
    return c.reshape(n, h, D // 2), s.reshape(n, h, D // GROUP[fmt])


def tokens(cache, pages, n, head):
    """(codes, scales) of one head's first n tokens: cache (codes, scales) [pages, heads, page, ...]."""
    return tuple(c[pages, head].reshape(-1, c.shape[-1])[:n] for c in cache)


def attention(q, k, v, fmt, pos, scale, window=0, T=None, kg=None, vg=None):
    """(out, bound) of queries q [m, D] at places pos [m] over one head's tokens, k and v
    (codes, scales) [L, ...]; T [D/G, G, G] transforms the queries."""
    D = q.shape[1]
    K, mag = weights(*k, fmt, kg), magnitudes(*k, fmt, kg)
    V = weights(*v, fmt, vg)
    dq = np.zeros_like(q)
    if T is not None:
        q, a = blocks(q, T)
        dq = T.shape[-1] * U * a + 2.0**-17 * np.abs(q)
    s = scale * (q @ K.T)
    ds = scale * ((D + 16) * U * (np.abs(q) @ mag.T) + dq @ mag.T)
    t = np.arange(K.shape[0])
    seen = t <= pos[:, None]
    if window:
        seen &= t > pos[:, None] - window
    none = ~seen.any(1, keepdims=True)
    s = np.where(seen, s, -np.inf)
    m = np.where(none, 0.0, s.max(1, keepdims=True, initial=-np.inf))
    with np.errstate(invalid="ignore"):
        gap = np.where(seen, np.abs(s - m), 0.0)
    p = np.where(seen, np.exp(s - m), 0.0)
    w = p / np.where(none, 1.0, p.sum(1, keepdims=True))
    out = w @ V
    # A probability: its score, the exponent's product and argument (the running maximum
    # may lie 2^8 below the largest), the exponential.
    dp = np.where(seen, ds + (4 * (gap + 16 + np.abs(m)) + 16) * U, 0.0)
    n = K.shape[0] + 64
    # Rounded probabilities, of which the denominator is the sum: w (1 + d), |d| <= e, move the
    # result by sum w d (V - out) / (1 + sum w d), at most e (w |V - out|) / (1 - e).  MXFP4
    # has them in bf16, the others in fp16, cut off at 2^-32 of the largest, as are INT4's
    # values, cut off at 2^-22.  fp32 sums; the denominator; the result.
    e = BF16 if fmt == "mxfp4" else 2.0**-11
    cut = 0.0 if fmt == "mxfp4" else 2.0**-32 * seen
    rel = e + (e if fmt == "int4" else 0) + n * U
    bound = (w * (dp + rel) + cut) @ np.abs(V) + (2.0**-22 if fmt == "int4" else 0)
    bound = bound + np.abs(out) * ((w * dp + cut).sum(1, keepdims=True) + e + n * U)
    return out, 1.05 * bound + BF16 * np.abs(out) + 1e-30
