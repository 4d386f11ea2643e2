"""Seeded caches, batches and their device tensors for the tests of the 4-bit cache."""

from __future__ import annotations

import numpy as np

from oracle import kv4 as ref
from tests.decode_cases import bf16, dev, dev_bf16, dev_scales, values, weights

GROUP = ref.GROUP


class Batch:
    """A cache with its pages in random order, and queries of every sequence."""

    def __init__(self, rng, fmt, D, heads, group, page, lengths, counts, T=False, width=None, spread=1.0):
        self.fmt, self.D, self.heads, self.group, self.page = fmt, D, heads, group, page
        self.lengths, self.counts = np.asarray(lengths, np.int32), np.asarray(counts, np.int32)
        need = [-(-int(n) // page) for n in lengths]
        self.pages = sum(need) + 3
        order = rng.permutation(self.pages).astype(np.int32)
        # Entries behind a sequence's last page are not read: no page at all.
        self.table = np.full((len(lengths), width or max(max(need), 1)), -12345, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at : at + n]
            at += n
        lead = (self.pages, heads, page)
        self.k, self.v = weights(rng, fmt, lead, D), weights(rng, fmt, lead, D)
        G = GROUP[fmt]
        if fmt == "nvfp4":  # finite scales only
            self.g = np.float32(2e-3), np.float32(3e-3)
        else:
            self.g = None, None
        # Scores of a few units.
        size = {"mxfp4": 0.03, "nvfp4": 0.3, "int4": 0.03}[fmt]
        self.n = int(self.counts.sum())
        self.q, self.q_bits = bf16(spread * rng.standard_normal((self.n, heads * group, D)) / size)
        self.T, self.T_bits = (bf16(rng.standard_normal((heads, D // G, G, G)) / G**0.5) if T else (None, None))
        self.start = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)
        self.scale = D**-0.5

    def cache(self):
        import mxfp4_activation_amd as wush

        gs = [None if g is None else dev(np.array([g])) for g in self.g]
        return wush.KV4Cache(dev(self.k[0]), dev_scales(self.fmt, self.k[1]), dev(self.v[0]),
                             dev_scales(self.fmt, self.v[1]), *gs)

    def run(self, cache=None, window=0, **kw):
        import mxfp4_activation_amd as wush

        return wush.kv4_attention(self.fmt, dev_bf16(self.q_bits), cache or self.cache(), dev(self.table),
                                  dev(self.lengths), q_start=dev(self.start), window=window,
                                  T_q=None if self.T is None else dev_bf16(self.T_bits), **kw)

    def want(self, window=0):
        """(out, bound) [n, q_heads, D]."""
        out = np.zeros_like(self.q)
        bound = np.zeros_like(self.q)
        for b, L in enumerate(self.lengths):
            lo, hi = self.start[b], self.start[b + 1]
            m = hi - lo
            pos = np.repeat(L - m + np.arange(m), self.group)
            pages = self.table[b, : -(-int(L) // self.page)]
            for h in range(self.heads):
                sl = slice(h * self.group, (h + 1) * self.group)
                k, v = (ref.tokens(c, pages, int(L), h) for c in (self.k, self.v))
                o, d = ref.attention(self.q[lo:hi, sl].reshape(-1, self.D), k, v, self.fmt, pos, self.scale, window,
                                     None if self.T is None else self.T[h], *self.g)
                out[lo:hi, sl] = o.reshape(m, self.group, self.D)
                bound[lo:hi, sl] = d.reshape(m, self.group, self.D)
        return out, bound

    def check(self, window=0, **kw):
        got = values(self.run(window=window, **kw))
        want, bound = self.want(window)
        off = np.abs(got - want) - bound
        assert np.all(off <= 0), (float(off.max()), np.unravel_index(int(off.argmax()), off.shape), int((off > 0).sum()))
        return got
