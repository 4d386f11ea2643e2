"""A paged cache of keys and values in 4 bits, and attention over it.

Like ``decode``, these functions only marshal arguments: they allocate outputs
and workspace with torch and enqueue the library call on torch's current stream.
Where it is built, native code does that (``_lib.binding``), and leaves to the
code here what is not plainly right.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .decode import _check, _check_global, _enter, _fmt, _scale_dtype, _workspace


class KV4Cache(NamedTuple):
    """One layer's keys and values: codes uint8 [pages, heads, page, D/2], scales
    [pages, heads, page, D/G] (uint8, or float16 for INT4), for NVFP4 the tensor
    scales (float32, one element each, not negative).  Token slot s is place s % page of
    page s // page; page is a power of two from 16 on, D 64, 128 or 256."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor
    k_global: Optional[torch.Tensor] = None
    v_global: Optional[torch.Tensor] = None


def kv4_cache(fmt: str, pages: int, heads: int, page: int, D: int, device="cuda",
              k_global: Optional[torch.Tensor] = None, v_global: Optional[torch.Tensor] = None) -> KV4Cache:
    """An unwritten cache."""
    _, G = _fmt(fmt)
    codes = [torch.empty((pages, heads, page, D // 2), dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.empty((pages, heads, page, D // G), dtype=_scale_dtype(fmt), device=device) for _ in range(2)]
    return KV4Cache(codes[0], scales[0], codes[1], scales[1], k_global, v_global)


def _heads(x: torch.Tensor, name: str):
    """(rows, heads, D, row stride) of a bf16 tensor [rows, heads, D] whose rows are contiguous."""
    if x.dtype != torch.bfloat16:
        raise TypeError("%s must be bfloat16 (got %s)" % (name, x.dtype))
    if x.dim() != 3:
        raise ValueError("%s must be [tokens, heads, D]" % name)
    n, h, D = x.shape
    if n and ((D > 1 and x.stride(2) != 1) or (h > 1 and x.stride(1) != D)):
        raise ValueError("%s must have contiguous rows [heads, D]" % name)
    return n, h, D, x.stride(0)


def _check_cache(fmt: str, c: KV4Cache, D: int, dev):
    """(addresses in the ABI's order, pages, heads, page, tensors to hold until the call)."""
    G = _fmt(fmt)[1]
    if not isinstance(c.k_codes, torch.Tensor) or c.k_codes.dim() != 4:
        raise ValueError("cache.k_codes must be a tensor [pages, heads, page, D/2]")
    pages, heads, page = c.k_codes.shape[:3]
    code, scale, sdt = (pages, heads, page, D // 2), (pages, heads, page, D // G), _scale_dtype(fmt)
    kc = _check(c.k_codes, "cache.k_codes", torch.uint8, code, dev)
    ks = _check(c.k_scales, "cache.k_scales", sdt, scale, dev)
    vc = _check(c.v_codes, "cache.v_codes", torch.uint8, code, dev)
    vs = _check(c.v_scales, "cache.v_scales", sdt, scale, dev)
    kg, hold_k = _check_global(fmt, c.k_global, "cache.k_global", 1, dev)
    vg, hold_v = _check_global(fmt, c.v_global, "cache.v_global", 1, dev)
    return (kc, ks, kg, vc, vs, vg), pages, heads, page, (hold_k, hold_v)


def _bank(T, name: str, heads: int, D: int, G: int, dev):
    return None if T is None else _check(T, name, torch.bfloat16, (heads, D // G, G, G), dev)


def kv4_append(fmt: str, k: torch.Tensor, v: torch.Tensor, cache: KV4Cache, slots: torch.Tensor,
               T_k: Optional[torch.Tensor] = None, T_v: Optional[torch.Tensor] = None) -> None:
    """Quantizes keys and values k, v [n, heads, D] (bf16, rows contiguous, any row
    stride that is a multiple of 8) into the cache's slots [n] (int64; outside the
    cache, a negative one say: not written; otherwise all different), after the
    block transforms T_k, T_v [heads, D/G, G, G], if given."""
    native = _lib.binding()
    if native is not None:
        st = native.append(fmt, k, v, *cache, slots, T_k, T_v)
        if st is not None:
            if st:
                _lib.check(st, "wush_kv4_append(%s)" % fmt)
            return
    f, G = _fmt(fmt)
    n, h, D, ldk = _heads(k, "k")
    dev, stream = _enter(k, "k")
    if v.shape != k.shape:
        raise ValueError("v must have the shape of k (got %s, %s)" % (tuple(v.shape), tuple(k.shape)))
    ldv = _heads(v, "v")[3]
    if v.device != dev:
        raise ValueError("v must be on %s (got %s)" % (dev, v.device))
    (kc, ks, kg, vc, vs, vg), pages, heads, page, hold = _check_cache(fmt, cache, D, dev)
    if heads != h:
        raise ValueError("the cache has %d heads, k has %d" % (heads, h))
    sl = _check(slots, "slots", torch.int64, (n,), dev)
    tk, tv = _bank(T_k, "T_k", h, D, G, dev), _bank(T_v, "T_v", h, D, G, dev)
    st = _lib.load().wush_kv4_append(f, k.data_ptr(), ldk, v.data_ptr(), ldv, tk, tv, sl, n, h, D, page, pages, kc, ks,
                                     kg, vc, vs, vg, stream)
    if st:
        _lib.check(st, "wush_kv4_append(%s)" % fmt)


def kv4_attention(fmt: str, q: torch.Tensor, cache: KV4Cache, block_table: torch.Tensor, lengths: torch.Tensor,
                  q_start: Optional[torch.Tensor] = None, scale: Optional[float] = None, window: int = 0,
                  T_q: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of queries q [n, q_heads, D] (bf16, as k in ``kv4_append``) over the
    cache: token t of sequence b is in page block_table[b, t // page] (int32 [B, width],
    rows contiguous), and lengths [B] (int32) counts its tokens, the queries' own
    included.  q_start [B + 1] (int32) gives each sequence's rows of q; without it each
    has one.  The last query of a sequence is its last token; a query sees the tokens
    up to its own, or the last `window` of them, and its result depends on those alone.
    scale: D ** -0.5 unless given.  T_q
    [heads, D/G, G, G] goes with keys that were transformed.  Returns bf16
    [n, q_heads, D]; rows from q_start[B] on are not written."""
    native = _lib.binding()
    if native is not None:
        r = native.attention(fmt, q, *cache, block_table, lengths, q_start, scale, window, T_q, out)
        if r is not None:
            if type(r) is int:
                _lib.check(r, "wush_kv4_attention(%s)" % fmt)
            return r
    f, G = _fmt(fmt)
    n, hq, D, ldq = _heads(q, "q")
    dev, stream = _enter(q, "q")
    (kc, ks, kg, vc, vs, vg), pages, heads, page, hold = _check_cache(fmt, cache, D, dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2 or block_table.dtype != torch.int32:
        raise TypeError("block_table must be an int32 tensor [B, width]")
    if block_table.device != dev:
        raise ValueError("block_table must be on %s (got %s)" % (dev, block_table.device))
    B, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table must have contiguous rows")
    pl = _check(lengths, "lengths", torch.int32, (B,), dev)
    pq = None if q_start is None else _check(q_start, "q_start", torch.int32, (B + 1,), dev)
    tq = _bank(T_q, "T_q", heads, D, G, dev)
    if out is None:
        out = torch.empty((n, hq, D), dtype=torch.bfloat16, device=dev)
        po = out.data_ptr()
    else:
        po = _check(out, "out", torch.bfloat16, (n, hq, D), dev)
    lib = _lib.load()
    nw = lib.wush_kv4_attention_workspace(f, B, n, hq, heads, D, page, width)
    ws = _workspace(nw, dev)
    st = lib.wush_kv4_attention(f, q.data_ptr(), ldq, tq, kc, ks, kg, vc, vs, vg, block_table.data_ptr(),
                                block_table.stride(0), width, pl, pq, B, n, hq, heads, D, page, pages,
                                D**-0.5 if scale is None else scale, window, po, ws.data_ptr() if nw else None, nw,
                                stream)
    if st:
        _lib.check(st, "wush_kv4_attention(%s)" % fmt)
    return out
