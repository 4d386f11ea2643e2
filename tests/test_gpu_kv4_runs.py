"""Attention whose items are cut: into equal runs of units, where a workgroup ends one item and
begins another, and into pieces of one item each, for every shape of workgroup."""

import numpy as np
import pytest

from oracle import kv4 as ref
from tests.decode_cases import FMTS, dev, dev_bf16, values
from tests.kv4_cases import Batch
from tests.kv4_shares import NARROW, PROMPT, WIDE, plan

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


def _plan(b, window):
    return plan(b.fmt, b.D, b.heads, b.group, b.page, b.table.shape[1], b.lengths, b.counts, window)


def _check_some(b, window, rng, pairs=14, queries=24):
    """Some of the queries (the first, the last and random ones) of some sequences and key heads, against float64."""
    got = values(b.run(window=window))
    assert np.isfinite(got).all()
    chosen = rng.permutation(len(b.lengths) * b.heads)[:pairs]
    for s, h in zip(chosen // b.heads, chosen % b.heads):
        L, c, lo = int(b.lengths[s]), int(b.counts[s]), int(b.start[s])
        if c == 0:
            continue
        i = np.unique(np.concatenate([[0, c - 1], rng.integers(0, c, size=queries)]))
        heads = slice(h * b.group, (h + 1) * b.group)
        k, v = (ref.tokens(x, b.table[s, : -(-L // b.page)], L, h) for x in (b.k, b.v))
        want, bound = ref.attention(b.q[lo + i][:, heads].reshape(-1, b.D), k, v, b.fmt, np.repeat(L - c + i, b.group), b.scale,
                                    window, None if b.T is None else b.T[h], *b.g)
        off = np.abs(got[lo + i][:, heads].reshape(-1, b.D) - want) - bound
        assert np.all(off <= 0), (s, h, float(off.max()), int((off > 0).sum()))


# Shape, D, key heads, queries per key head, page, sequences, their tokens, their queries.
_RUNS = [
    (NARROW, 64, 4, 4, 32, 60, (5000, 9000), (1, 2)),
    (NARROW, 128, 4, 2, 64, 48, (5000, 9500), (1, 1)),
    (NARROW, 256, 2, 4, 16, 44, (6000, 9500), (1, 7)),
    (WIDE, 64, 4, 4, 16, 40, (6500, 9500), (4, 8)),
    (WIDE, 128, 2, 5, 128, 44, (6500, 9500), (4, 9)),
    (PROMPT, 64, 4, 2, 64, 4, (17000, 23000), (130, 170)),
    (PROMPT, 128, 2, 4, 32, 4, (18000, 24000), (100, 160)),
    (PROMPT, 256, 2, 3, 64, 3, (18000, 23000), (90, 130)),
]


def _batch(rng, fmt, case, T=False, scale=1.0):
    _, D, heads, group, page, B, tokens, queries = case
    lengths = (rng.integers(*tokens, size=B, endpoint=True) * scale).astype(int)
    return Batch(rng, fmt, D, heads, group, page, lengths, rng.integers(*queries, size=B, endpoint=True), T=T)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [False, True])
@pytest.mark.parametrize("case", _RUNS, ids=lambda c: "%s-%d" % (("narrow", "wide", "prompt")[c[0]], c[1]))
def test_equal_runs(fmt, T, case):
    rng = np.random.default_rng(case[1] + case[0])
    b = _batch(rng, fmt, case, T)
    p = _plan(b, 0)
    assert p.by_runs and p.shape == case[0], p
    _check_some(b, 0, rng)


@pytest.mark.parametrize("fmt,case,sequences,window", [
    ("nvfp4", _RUNS[0], 160, 5000), ("int4", _RUNS[1], 150, 6001), ("mxfp4", _RUNS[4], 70, 6400), ("mxfp4", _RUNS[6], 8, 15000),
    ("int4", _RUNS[7], 8, 11111)], ids=str)
def test_equal_runs_of_windows(fmt, case, sequences, window):
    rng = np.random.default_rng(window)
    b = _batch(rng, fmt, (*case[:5], sequences, *case[6:]))
    p = _plan(b, window)
    assert p.by_runs and p.shape == case[0], (p.shape, p.share, p.whole)
    _check_some(b, window, rng)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", [_RUNS[4], _RUNS[6]], ids=["wide", "prompt"])
def test_pieces_of_one_item_with_transforms(fmt, case):
    rng = np.random.default_rng(3)
    b = _batch(rng, fmt, case, T=True, scale=0.2)
    p = _plan(b, 0)
    assert not p.by_runs and not p.whole and max(p.units) > p.share and p.shape == case[0], p
    _check_some(b, 0, rng)


@pytest.mark.parametrize("fmt,case", [("mxfp4", _RUNS[1]), ("int4", _RUNS[4]), ("nvfp4", _RUNS[6])], ids=["narrow", "wide", "prompt"])
def test_a_bad_page_among_equal_runs(fmt, case):
    """Its sequence is NaN; the others are what they are, bit for bit."""
    rng = np.random.default_rng(5)
    b = _batch(rng, fmt, case)
    assert _plan(b, 0).by_runs
    good = b.run()
    for s, page in ((1, -1), (2, b.pages)):
        table = b.table.copy()
        table[s, 30] = page
        kept, b.table = b.table, table
        got = b.run()
        b.table = kept
        lo, hi = b.start[s], b.start[s + 1]
        assert torch.isnan(got[lo:hi]).all()
        assert torch.equal(got[:lo], good[:lo]) and torch.equal(got[hi:], good[hi:])


@pytest.mark.parametrize("fmt,case", [("int4", _RUNS[1]), ("nvfp4", _RUNS[4]), ("mxfp4", _RUNS[6])], ids=["narrow", "wide", "prompt"])
def test_graph_replays_between_runs_and_pieces(fmt, case):
    """One captured call, replayed with lengths by which its items are in runs, in pieces and whole."""
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(6)
    b = _batch(rng, fmt, case)
    full = b.lengths.copy()
    q, cache, table, lengths, start = dev_bf16(b.q_bits), b.cache(), dev(b.table), dev(full), dev(b.start)
    out = torch.empty_like(q)
    call = lambda: wush.kv4_attention(fmt, q, cache, table, lengths, q_start=start, out=out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    ways = set()
    for scale in (1.0, 0.25, 0.02, 1.0, 0.25):
        b.lengths = np.maximum((full * scale).astype(np.int32), 1)
        p = _plan(b, 0)
        ways.add("runs" if p.by_runs else "whole" if p.whole else "pieces")
        lengths.copy_(dev(b.lengths))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        assert torch.isfinite(replayed).all()
        assert torch.equal(call().clone(), replayed)
    assert {"runs", "pieces"} <= ways


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", [_RUNS[1], _RUNS[4], _RUNS[6]], ids=["narrow", "wide", "prompt"])
@pytest.mark.parametrize("window", [0, 4000])
def test_values_that_are_not_finite_among_runs(fmt, case, window):
    """They spoil their group's channels for the queries that see them; everything else stays, bit for bit."""
    rng = np.random.default_rng(8)
    case = (*case[:7], (2, 3)) if case[0] == NARROW else case  # several queries, so that some do not see it
    b = _batch(rng, fmt, case)
    assert _plan(b, 0).by_runs and _plan(b, 0).shape == case[0]
    good = b.run(window=window)
    G = 16 if fmt == "nvfp4" else 32
    hit = np.zeros((b.n, b.heads * b.group, b.D), bool)
    for s in range(0, len(b.lengths), 2):
        L, c = int(b.lengths[s]), int(b.counts[s])
        for at in (L - 1, L - 1 - c // 2, L - c - 2500, 40):
            page, place, g = b.table[s, at // b.page], at % b.page, int(rng.integers(0, b.D // G))
            b.v[1][page, :, place, g] = {"mxfp4": 0xFF, "nvfp4": 0x7F, "int4": 0x7C00}[fmt]
            b.v[0][page, :, place, g * G // 2 : (g + 1) * G // 2] = 0x77
            pos = L - c + np.arange(c)
            rows = b.start[s] + np.nonzero((at <= pos) & ((window == 0) | (at > pos - window)))[0]
            hit[rows, :, g * G : (g + 1) * G] = True
    got, hit = b.run(window=window), torch.from_numpy(hit).cuda()
    assert torch.equal(got[~hit], good[~hit]) and not torch.isfinite(got[hit]).any()
