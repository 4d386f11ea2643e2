"""Float64 definitions of the decode operators, with error bounds.

Linear layers and mixtures of experts on 4-bit weights, and token log
probabilities, for the parity tests.  Each function that computes sums also
returns a bound on what a correct fp32 evaluation may differ by, from these
rules (u = 2^-23, one fp32 rounding or truncation):

* a sum of n products that are exact in fp32 errs by at most n u sum |terms|, in
  any order (n - 1 additions, each off by at most u of a partial sum);
* INT4 codes enter as code + 8 with -8 sum x in the same sum, so its terms are
  (code + 8) x and 8 x, and the group's fp32 scale adds one rounding;
* an operand kept as two bf16 planes is off by at most 2^-17 of itself, as
  three planes by at most u;
* exp, the logarithm and the division of one value: 8 u relative, plus u
  times the exponent's argument.
"""

from __future__ import annotations

import numpy as np

from . import codecs

GROUP = {"mxfp4": 32, "nvfp4": 16, "int4": 32}
U = 2.0**-23


def _split(codes, scales, fmt):
    """(element values, scales per element) of codes [..., K/2], scales [..., K/G]."""
    nib = codecs.unpack_nibbles(codes)
    v = codecs.int4_decode(nib).astype(np.float64) if fmt == "int4" else codecs.e2m1_decode(nib).astype(np.float64)
    if fmt == "mxfp4":
        s = codecs.e8m0_value(scales)
    elif fmt == "nvfp4":
        s = codecs.e4m3_value(scales)
    else:
        s = scales.view(np.float16).astype(np.float64)
    return v, np.repeat(s, GROUP[fmt], axis=-1)


def weights(codes, scales, fmt, global_scale=None):
    """The values of 4-bit weights [..., K]; global_scale broadcasts over them."""
    v, s = _split(codes, scales, fmt)
    w = v * s
    return w if global_scale is None else w * global_scale


def magnitudes(codes, scales, fmt, global_scale=None):
    """Per weight, the magnitude of the terms it enters the fp32 sum with."""
    v, s = _split(codes, scales, fmt)
    m = (np.abs(v + 8) + 8 if fmt == "int4" else np.abs(v)) * s
    return m if global_scale is None else m * global_scale


def blocks(x, T):
    """(T x per block of the last axis, sum |T x| terms)."""
    C, G = T.shape[-3], T.shape[-1]
    xb = x.reshape(x.shape[:-1] + (C, G, 1))
    y = np.matmul(T, xb)[..., 0]
    a = np.matmul(np.abs(T), np.abs(xb))[..., 0]
    return y.reshape(x.shape), a.reshape(x.shape)


def linear(x, codes, scales, fmt, T=None, global_scale=None, planes=2):
    """(x' W^T, bound) for x [M, K]."""
    K = x.shape[-1]
    w, mag = weights(codes, scales, fmt, global_scale), magnitudes(codes, scales, fmt, global_scale)
    dx = np.zeros_like(x)
    if T is not None:
        x, a = blocks(x, T)
        dx = T.shape[-1] * U * a + (2.0**-17 if planes == 2 else U) * np.abs(x)
    return x @ w.T, (K + 8) * U * (np.abs(x) @ mag.T) + dx @ mag.T


def choose(logits, topk, renormalize):
    """(ids, weights): the topk largest per row, ties to the lower index."""
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :topk]
    e = np.exp(logits - logits.max(1, keepdims=True))
    p = np.take_along_axis(e, ids, 1)
    return ids, p / (p if renormalize else e).sum(1, keepdims=True)


def moe(x, router, gate_up, down, topk, renormalize, fmt, planes=2):
    """(y, bound, ids, weights).  gate_up and down: (codes, scales, global
    scales [E] or None, transforms or None)."""
    logits = x @ router.T
    d_logit = x.shape[1] * U * (np.abs(x) @ np.abs(router).T).max()
    ids, w = choose(logits, topk, renormalize)
    y, bound = np.zeros_like(x), np.zeros_like(x)
    for e in np.unique(ids):
        m, j = np.nonzero(ids == e)
        gs = lambda p: None if p[2] is None else p[2][e]  # noqa: E731
        gu, d_gu = linear(x[m], gate_up[0][e], gate_up[1][e], fmt, gate_up[3], gs(gate_up), planes)
        I = gu.shape[1] // 2
        g, u, dg, du = gu[:, :I], gu[:, I:], d_gu[:, :I], d_gu[:, I:]
        s = g / (1 + np.exp(-g))
        h = s * u
        # |silu'| <= 1.1; one exponential, one division, two products.
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + (20 + np.abs(g)) * U * np.abs(h)
        if down[3] is not None:
            T = down[3][e]
            h, a = blocks(h, T)
            dh = blocks(dh, np.abs(T))[0] + T.shape[-1] * U * a
        dh = dh + (2.0**-17 if planes == 2 else U) * np.abs(h)
        wd = weights(down[0][e], down[1][e], fmt, gs(down))
        mag = magnitudes(down[0][e], down[1][e], fmt, gs(down))
        o = h @ wd.T
        do = dh @ mag.T + (I + 8) * U * (np.abs(h) @ mag.T)
        c = w[m, j][:, None]
        y[m] += c * o
        # The weight: two exponentials' arguments off by d_logit, sums and a division.
        bound[m] += c * do + c * np.abs(o) * (4 * d_logit + (40 + topk) * U)
    return y, bound + 8 * U * np.abs(y), ids, w


def token_logprobs(logits, targets, top):
    """(logprob, entropy, ids, top logprobs, bound per row) with the library's
    conventions for masked, empty and unscored rows; NaN rows are the caller's."""
    R, V = logits.shape
    m = logits.max(1, keepdims=True)
    empty = np.isneginf(m[:, 0])
    d = logits - np.where(np.isneginf(m), 0.0, m)
    e = np.exp(d)
    S = np.where(empty, 1.0, e.sum(1))
    z = np.where(e > 0, e * np.where(e > 0, d, 0.0), 0.0)
    mean = np.where(empty, 0.0, z.sum(1) / S)
    entropy = np.where(empty, 0.0, np.log(S) - mean)
    lp = np.where(empty[:, None], -np.inf, d - np.log(S)[:, None])
    score = lp[np.arange(R), np.clip(targets, 0, V - 1)]
    score = np.where(targets < 0, 0.0, np.where(targets >= V, np.nan, score))
    n = min(top, V)
    order = np.argsort(-logits, axis=1, kind="stable")[:, :n]
    alt = np.take_along_axis(lp, order, 1)
    ids = np.where(np.isneginf(alt), -1, order)
    pad = ((0, 0), (0, top - n))
    ids, alt = np.pad(ids, pad, constant_values=-1), np.pad(alt, pad, constant_values=-np.inf)
    # Each thread adds about V / 256 terms and joins a few dozen partial sums; every
    # term's exponent is off by u |d|, which enters weighed by its probability.
    n_sum = V / 256 + 96
    bound = U * (n_sum * (1 + np.abs(mean)) + 8 * (1 + np.abs(mean)) + 4 * np.log(S))
    second = np.where(empty, 0.0, (z * np.where(e > 0, d, 0.0)).sum(1) / S)
    return score, entropy, ids, alt, bound + 4 * U * second
