"""GPU parity of the token log probabilities (wush_token_logprobs) with the
float64 oracle: ids must match exactly, values within the oracle's bound of the
fp32 sums plus the rounding of the results themselves."""

import numpy as np
import pytest

from oracle import codecs, decode
from synthetic import f64_to_bf16_bits
from tests import decode_cases as dc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


def _typed(l, dtype):
    """(float64 values after rounding, device tensor)."""
    if dtype == "bf16":
        b = f64_to_bf16_bits(l)
        return codecs.bf16_bits_to_f32(b).astype(np.float64), dc.dev_bf16(b)
    v = l.astype(np.float16 if dtype == "f16" else np.float32)
    return v.astype(np.float64), dc.dev(v)


def _close(got, want, bound):
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        err = np.where(same, 0.0, np.abs(got - want))
    assert np.all(err <= bound), np.nanmax(err / bound)


def _check(l, dev_l, targets, top):
    import mxfp4_activation_amd as wush

    got = wush.token_logprobs(dev_l, dc.dev(targets), top=top)
    score, entropy, ids, alt, bound = decode.token_logprobs(l, targets, top)
    assert np.array_equal(got.top_ids.cpu().numpy(), ids)
    fin = np.where(np.isfinite(score), np.abs(score), 0.0)
    _close(dc.values(got.logprob), score, bound + 4 * decode.U * fin)
    _close(dc.values(got.entropy), entropy, bound + 4 * decode.U * entropy)
    fin = np.where(np.isfinite(alt), np.abs(alt), 0.0)
    _close(dc.values(got.top_logprobs), alt, bound[:, None] + 4 * decode.U * fin)
    return got


# Vocabularies around the vectors (4, 8), a thread's share (32), a workgroup's
# batch (8192) and several batches; one row and many (split and whole rows).
@pytest.mark.parametrize("top", [0, 1, 20, 32])
@pytest.mark.parametrize("R,V", [(1, 1), (2, 7), (3, 33), (5, 1000), (1, 8192), (2, 8193), (1, 50001), (1100, 300),
                                 (1030, 9001), (4, 140000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_parity(dtype, R, V, top):
    if R > 1000 and (dtype == "f16" or top == 1):
        pytest.skip("covered by the other types and lengths")
    rng = np.random.default_rng(R + V)
    l, d = _typed(rng.standard_normal((R, V)) * 3, dtype)
    _check(l, d, rng.integers(0, V, size=R), top)


@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 5), (13, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_any_stride_and_start(dtype, pad, offset):
    """Rows off every vector boundary; NaN around the rows must not be read as theirs."""
    rng = np.random.default_rng(pad)
    R, V = 6, 8200
    big = np.full((R, V + pad + offset), np.nan)
    big[:, offset : offset + V] = rng.standard_normal((R, V)) * 2
    l, d = _typed(np.nan_to_num(big, nan=0.0), dtype)
    d.view(R, -1)[:, :offset] = float("nan")
    d.view(R, -1)[:, offset + V :] = float("nan")
    _check(l[:, offset : offset + V], d[:, offset : offset + V], rng.integers(0, V, size=R), 5)


@pytest.mark.parametrize("V", [100, 20000])
def test_masks(V):
    rng = np.random.default_rng(1)
    R = 8
    l = rng.standard_normal((R, V)) * 3
    l[0, :] = -INF  # nothing left
    l[1, 1:] = -INF  # one token
    l[2, : V // 2] = -INF
    l[3, rng.random(V) < 0.98] = -INF
    l[4, :] = np.finfo(np.float32).min  # the type's lowest value masks nothing by itself
    l[5, 3:] = np.finfo(np.float32).min
    l[6, V - 2 :] = 40.0
    l, d = _typed(l, "f32")
    got = _check(l, d, np.array([3, 0, V - 1, 5, 9, 1, V - 1, -100]), 7)
    assert got.entropy[0] == 0 and got.logprob[0] == -INF and torch.all(got.top_ids[0] == -1)
    assert got.logprob[1] == 0 and got.entropy[1] == 0
    assert got.logprob[7] == 0


@pytest.mark.parametrize("R", [2, 600])
def test_order_of_equal_and_sorted_rows(R):
    """All equal, rising, falling, few distinct values: the lowest ids win,
    however the candidates fall on threads, waves and batches."""
    V = 30000
    rng = np.random.default_rng(2)
    kinds = [np.zeros(V), np.arange(V) / 256.0, -np.arange(V) / 256.0, rng.integers(0, 3, V).astype(float),
             np.where(np.arange(V) % 2048 < 8, 5.0, 0.0), np.where(np.arange(V) // 2048 == 2, 5.0, 0.0)]
    l, d = _typed(np.stack([kinds[i % len(kinds)] for i in range(max(R, 6))]), "f32")
    _check(l, d, rng.integers(0, V, size=l.shape[0]), 32)


def test_nan_and_infinity_rows():
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(3)
    for V in (50, 20000):
        l = rng.standard_normal((6, V)).astype(np.float32)
        l[1, V // 3] = np.nan
        l[2, :] = np.nan
        l[3, V - 1] = np.inf
        l[4, :] = -np.inf
        l[4, 7] = np.nan
        got = wush.token_logprobs(dc.dev(l), dc.dev(np.array([0, 0, 0, 0, 0, V])), top=3)
        for r in (1, 2, 3, 4):
            assert torch.isnan(got.logprob[r]) and torch.isnan(got.entropy[r])
            assert torch.all(got.top_ids[r] == -1) and torch.isnan(got.top_logprobs[r]).all()
        assert torch.isfinite(got.logprob[0]) and torch.isfinite(got.top_logprobs[0]).all()
        assert torch.isnan(got.logprob[5]) and torch.isfinite(got.entropy[5])  # no such token


def test_confident_rows_keep_their_digits():
    """A row whose mass sits on one token: log p and entropy near zero."""
    l = np.full((2, 1000), -30.0)
    l[:, 4] = 0.0
    l, d = _typed(l, "f32")
    _check(l, d, np.array([4, 5]), 2)


def test_graph_replay_side_stream_and_empty():
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(4)
    sets = [_typed(rng.standard_normal((3, 40000)), "bf16")[1] for _ in range(3)]
    t = dc.dev(np.array([1, 2, 39999]))
    eager = [wush.token_logprobs(s, t, top=4) for s in sets]
    x = sets[0].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = wush.token_logprobs(x, t, top=4)
    for turn in (0, 1, 2, 1):
        x.copy_(sets[turn])
        graph.replay()
        for a, b in zip(got, eager[turn]):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
    none = wush.token_logprobs(sets[0][:0], t[:0], top=4)
    assert none.logprob.shape == (0,) and none.top_ids.shape == (0, 4)
