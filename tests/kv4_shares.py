"""How kv4_attention shares its work out, restated on the host: for tests that are about one way
of doing so, and for the test of the rule itself.  The rule's constants are read from the
sources, the number of runs from the library's own workspace query."""

from __future__ import annotations

import os
import re
from typing import NamedTuple

import mxfp4_activation_amd as wush
from mxfp4_activation_amd import _lib

_CSRC = os.path.join(os.path.dirname(os.path.abspath(wush.__file__)), "csrc")


def _constant(name, file):
    with open(os.path.join(_CSRC, file)) as f:
        return float(re.search(r"constexpr \w+ %s = ([\d.]+)f?;" % name, f.read())[1])


UNIT = int(_constant("kKvUnit", "wush_kv4.h"))
RUN_UNITS = _constant("kRunUnits", "wush_kv4_attention.h")
JOIN_UNITS = _constant("kJoinUnits", "wush_kv4_attention.h")
ALONE_UNITS = _constant("kAloneUnits", "wush_kv4_attention.h")
JOIN_BYTES = 32
NARROW, WIDE, PROMPT = range(3)


def columns(shape, D):
    return 16 * (1 if shape == NARROW or D > 128 else 2) * (4 if shape == PROMPT else 1)


class Plan(NamedTuple):
    shape: int
    runs: int       # 0: nothing may be cut
    most: int       # items that the workspace has room for
    units: list     # of every item, in the kernel's order
    whole: bool     # every item is one piece
    share: int
    by_runs: bool


def plan(fmt, D, heads, group, page, width, lengths, counts, window=0) -> Plan:
    B, n = len(lengths), int(sum(counts))
    mean = n * group // B
    shape = NARROW if mean <= (32 if D > 128 else 16) else WIDE if mean <= 64 and D <= 128 else PROMPT
    nc = columns(shape, D)
    most = (n * group // nc + min(B, n)) * heads
    ws = wush.load().wush_kv4_attention_workspace(_lib.FMT[fmt], B, n, heads * group, heads, D, page, width)
    piece = 4 * nc * (D + 2)
    runs = max(ws - JOIN_BYTES * (1 + most), 0) // (2 * piece)
    assert ws == (JOIN_BYTES * (1 + most) + 2 * runs * piece if ws else 0)
    units = []
    for c, L in zip(counts, lengths):
        c, L, of = int(c), int(L), []
        for t in range(-(-c * group // nc)):
            i0, i1 = t * nc // group, min((t * nc + nc - 1) // group, c - 1)
            hi, lo = max(0, L - c + i1 + 1), max(0, L - c + i0 - window + 1) if window else 0
            of.append(-(-hi // UNIT) - lo // UNIT if hi > lo else 1)
        units += of * heads
    total = sum(units)
    if not runs:
        return Plan(shape, 0, most, units, True, 0, False)
    meeting = 0 if shape == PROMPT else JOIN_UNITS * runs
    if max(units) * -(-len(units) // runs) * runs <= 1.1 * total + meeting:
        return Plan(shape, runs, most, units, True, 0, False)
    share = -(-total // runs)
    if shape != PROMPT:
        share = max(share, min(int(ALONE_UNITS), -(-total // 256)))
    return Plan(shape, runs, most, units, False, share, share >= RUN_UNITS)
