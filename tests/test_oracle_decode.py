"""Pins of the decode oracle: each function against element-wise loops or
hand-made cases (CPU)."""

import math

import numpy as np
import pytest

from oracle import codecs, decode


def _rand_weights(rng, fmt, rows, K):
    codes = rng.integers(0, 256, size=(rows, K // 2), dtype=np.uint8)
    n = K // decode.GROUP[fmt]
    if fmt == "mxfp4":
        return codes, rng.integers(120, 134, size=(rows, n), dtype=np.uint8)
    if fmt == "nvfp4":
        return codes, rng.integers(0, 127, size=(rows, n), dtype=np.uint8)
    return codes, rng.random((rows, n)).astype(np.float16).view(np.uint16)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "int4"])
def test_linear_against_loops(fmt):
    rng = np.random.default_rng(3)
    M, N, G = 2, 3, decode.GROUP[fmt]
    K = 3 * G
    codes, scales = _rand_weights(rng, fmt, N, K)
    x = rng.standard_normal((M, K))
    T = rng.standard_normal((K // G, G, G))
    y, bound = decode.linear(x, codes, scales, fmt, T, 0.5)
    levels = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for m in range(M):
        for n in range(N):
            total = 0.0
            for k in range(K):
                nib = int(codes[n, k // 2]) >> (4 * (k % 2)) & 15
                if fmt == "int4":
                    v = (nib - 16 if nib >= 8 else nib) * float(scales[n, k // G : k // G + 1].view(np.float16)[0])
                else:
                    v = (-1 if nib & 8 else 1) * levels[nib & 7]
                    s = int(scales[n, k // G])
                    v *= 2.0 ** (s - 127) if fmt == "mxfp4" else float(codecs.e4m3_value(s))
                c, i = divmod(k, G)
                total += 0.5 * v * sum(T[c, i, j] * x[m, c * G + j] for j in range(G))
            assert y[m, n] == pytest.approx(total, rel=1e-12, abs=1e-12)
    assert np.all(bound > 0)


def test_choose_breaks_ties_to_the_lower_index():
    l = np.array([[1.0, 3.0, 3.0, 0.0, 3.0], [2.0, 2.0, 2.0, 2.0, 2.0]])
    ids, w = decode.choose(l, 3, True)
    assert ids.tolist() == [[1, 2, 4], [0, 1, 2]]
    assert np.allclose(w, 1 / 3)
    _, w = decode.choose(l, 3, False)
    assert w[1].tolist() == pytest.approx([0.2, 0.2, 0.2])


def test_moe_against_its_formula():
    rng = np.random.default_rng(4)
    M, E, H, I, k = 3, 4, 32, 32, 2
    gc, gsc = _rand_weights(rng, "mxfp4", E * 2 * I, H)
    dc, dsc = _rand_weights(rng, "mxfp4", E * H, I)
    gu = (gc.reshape(E, 2 * I, -1), gsc.reshape(E, 2 * I, -1) - 6, None, rng.standard_normal((1, 32, 32)))
    dn = (dc.reshape(E, H, -1), dsc.reshape(E, H, -1) - 6, None, rng.standard_normal((E, 1, 32, 32)))
    x, router = rng.standard_normal((M, H)), rng.standard_normal((E, H))
    y, bound, ids, w = decode.moe(x, router, gu, dn, k, True, "mxfp4")
    for m in range(M):
        want = np.zeros(H)
        for j in range(k):
            e = ids[m, j]
            W = decode.weights(gu[0][e], gu[1][e], "mxfp4")
            a = W @ (gu[3][0] @ x[m])
            h = np.array([g / (1 + math.exp(-g)) * u for g, u in zip(a[:I], a[I:])])
            want += w[m, j] * (decode.weights(dn[0][e], dn[1][e], "mxfp4") @ (dn[3][e][0] @ h))
        assert np.allclose(y[m], want, rtol=1e-10, atol=1e-10 * np.abs(want).max())
    assert np.all(bound >= 0)


def test_token_logprobs_against_loops():
    inf = math.inf
    l = np.array([[0.0, math.log(2), math.log(2), -inf], [-inf, -inf, -inf, -inf], [5.0, -inf, -inf, -inf]])
    t = np.array([1, 2, -1])
    lp, ent, ids, alt, _ = decode.token_logprobs(l, t, 6)
    p = np.array([0.2, 0.4, 0.4])
    assert lp.tolist() == pytest.approx([math.log(0.4), -inf, 0.0])
    assert ent.tolist() == pytest.approx([-(p * np.log(p)).sum(), 0.0, 0.0])
    assert ids.tolist() == [[1, 2, 0, -1, -1, -1], [-1] * 6, [0] + [-1] * 5]
    assert alt[0, :3].tolist() == pytest.approx([math.log(0.4), math.log(0.4), math.log(0.2)])
    assert np.isneginf(alt[1]).all() and alt[2, 0] == 0.0
    assert math.isnan(decode.token_logprobs(l[:1], np.array([4]), 0)[0][0])
