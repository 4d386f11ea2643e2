"""The runs by which attention's units are shared out, walked on the host as the kernel walks
them: every unit is done once, every piece has a place of its own in the workspace, and the
entries for joining name an item's pieces in order (CPU)."""

import random

import pytest

from tests.kv4_shares import PROMPT, RUN_UNITS, columns, plan


def _walk(p):
    """({place: (item, first unit, units)}, {entry: (item, places)}) of a plan by runs."""
    places, joins, whole = {}, {}, set()
    ranks, several = [], 0
    for u in p.units:
        ranks.append(several)
        several += u > 1
    starts = [0]
    for u in p.units:
        starts.append(starts[-1] + u)
    item = 0
    for w in range(p.runs):
        begin = w * p.share
        left = min(p.share, starts[-1] - begin)
        if left <= 0:
            continue
        while starts[item + 1] <= begin:
            item += 1
        i, off, slot = item, begin - starts[item], 2 * w
        while True:
            take = min(p.units[i] - off, left)
            left -= take
            rest = p.units[i] - off - take
            if take == p.units[i]:
                assert i not in whole
                whole.add(i)
            else:
                assert slot not in places
                places[slot] = (i, off, take)
            if p.units[i] > 1 and off == 0:
                pieces = (rest - 1) // p.share + 2 if rest > 0 else 0
                assert ranks[i] not in joins
                joins[ranks[i]] = (i, [slot] + [2 * w + 2 + 2 * k for k in range(pieces - 1)] if pieces else [])
            if left == 0:
                break
            i, off, slot = i + 1, 0, 2 * w + 1
    return places, joins, whole, several


@pytest.mark.parametrize("seed", range(40))
def test_runs_cover_the_units_and_fit_the_workspace(seed):
    rng = random.Random(seed)
    found = 0
    while not found:
        fmt, D = rng.choice(("mxfp4", "nvfp4", "int4")), rng.choice((64, 128, 256))
        B, heads, group, page = rng.choice((1, 3, 12, 70, 200)), rng.choice((1, 2, 8)), rng.choice((1, 4, 7)), 64
        most = rng.choice((1, 3, 30, 300))
        counts = [rng.randint(0, most) for _ in range(B)]
        if sum(counts) == 0:
            continue
        width = rng.choice((300, 2000))
        long = rng.choice((10, 2, 1))
        lengths = [rng.randint(0, width * page // (1 if rng.random() < 0.5 else long)) for _ in range(B)]
        p = plan(fmt, D, heads, group, page, width, lengths, counts, rng.choice((0, 0, 9000)))
        if not p.by_runs:
            continue
        found = 1
        assert p.share >= RUN_UNITS and len(p.units) <= p.most and p.share * p.runs >= sum(p.units)
        places, joins, whole, several = _walk(p)
        assert sorted(joins) == list(range(several)) and several <= p.most
        assert all(0 <= s < 2 * p.runs for s in places)
        parts = {}
        for slot, (i, off, take) in places.items():
            parts.setdefault(i, []).append((off, take, slot))
        assert whole | set(parts) == set(range(len(p.units))) and not whole & set(parts)
        named = {i: slots for i, slots in joins.values()}
        for i, of in parts.items():
            of.sort()
            at = 0
            for off, take, _ in of:
                assert off == at and take > 0
                at += take
            assert at == p.units[i] and named[i] == [slot for _, _, slot in of]
        assert all(named.get(i, []) == [] for i in whole)


def test_shapes_go_by_the_mean_of_columns():
    """(128 columns to a prompt's workgroup, 64 for heads of 256.)"""
    for D, counts, shape, cols in ((128, [16], 0, 16), (128, [17], 1, 32), (128, [65], 2, 128), (256, [32], 0, 16), (256, [33], 2, 64)):
        p = plan("mxfp4", D, 1, 1, 16, 100, [1000], counts)
        assert p.shape == shape and columns(shape, D) == cols
    assert PROMPT == 2
