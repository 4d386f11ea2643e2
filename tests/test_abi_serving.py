"""Refusals of the cache, attention, adapter and logit entries: the C ABI with fake
device addresses, before any HIP call, and the Python wrappers on host tensors (no
GPU needed); and what the shares of attention's work come to, against its workspace."""

import random

import pytest

import mxfp4_activation_amd as wush
from mxfp4_activation_amd import _lib

A = 1 << 40  # fake device address: never dereferenced
EINVAL, EALIGN, EUNSUPPORTED, OK = _lib.WUSH_EINVAL, _lib.WUSH_EALIGN, _lib.WUSH_EUNSUPPORTED, _lib.WUSH_OK


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_kv4_refusals(fmt):
    lib = wush.load()

    def append(fmt=fmt, n=2, heads=2, D=128, page=16, pages=4, K=A, ldk=256, slots=A * 3, kc=A * 10, kg=A * 12):
        return lib.wush_kv4_append(fmt, K, ldk, A * 2, 256, None, None, slots, n, heads, D, page, pages, kc, A * 11, kg,
                                   A * 13, A * 14, A * 15, None)

    assert append(n=0) == OK and append(pages=0) == OK
    assert append(fmt=4) == EUNSUPPORTED and append(D=80) == EUNSUPPORTED
    assert append(page=20) == EINVAL and append(heads=0) == EINVAL and append(slots=None) == EINVAL
    assert append(kc=A * 10 + 8) == EALIGN and append(ldk=260) == EALIGN and append(kc=A) == EINVAL
    if fmt == 1:
        assert append(kg=None) == EINVAL and b"global_scale" in lib.wush_last_error()

    def attend(fmt=fmt, Q=A, B=2, n=2, hq=8, h=2, scale=0.1, window=0, out=A * 5, ws=A * 6, need=1 << 40, start=None,
               width=40):
        return lib.wush_kv4_attention(fmt, Q, 1024, None, A * 10, A * 11, A * 12, A * 13, A * 14, A * 15, A * 3, width,
                                      width, A * 4, start, B, n, hq, h, 128, 16, 9, scale, window, out, ws, need, None)

    assert attend(B=0, n=0) == OK
    assert attend(scale=0.0) == EINVAL and attend(scale=float("nan")) == EINVAL and attend(window=-1) == EINVAL
    assert attend(hq=9) == EINVAL and attend(n=3) == EINVAL and attend(out=None) == EINVAL
    assert attend(need=8) == EINVAL and b"workspace" in lib.wush_last_error()
    assert attend(out=A * 5 + 4) == EALIGN and attend(out=A) == EINVAL and attend(ws=A * 5) == EINVAL


def test_lora_and_adjust_refusals():
    lib = wush.load()

    def lora(r=16, a=A * 5, ids=A * 8, n=1 << 40, Y=A * 9):
        return lib.wush_linear_w4_lora(0, A, 64, None, A * 2, A * 3, None, a, A * 6, A * 7, ids, 4, r, 2, 40, 64, Y, 0,
                                       A * 11, n, None)

    assert lora(r=12) == EINVAL and lora(r=1024) == EINVAL and lora(a=None) == EINVAL and lora(ids=None) == EINVAL
    assert lora(n=64) == EINVAL and lora(a=A * 5 + 2) == EALIGN and lora(Y=A * 6) == EINVAL

    def adjust(t=0, R=2, V=50, n=4, out=A * 9, ld=50):
        return lib.wush_adjust_logits(A, t, ld, R, V, A * 2, n, A * 3, n, A * 4, A * 5, A * 6, A * 7, A * 8, n, None, out,
                                      50, None)

    assert adjust(R=0) == OK
    assert adjust(t=9) == EINVAL and adjust(V=0) == EINVAL and adjust(ld=49) == EINVAL and adjust(out=A + 4) == EINVAL
    assert adjust(out=A * 9 + 2) == EALIGN and adjust(out=A * 8) == EINVAL


def test_wrappers_refuse():
    torch = pytest.importorskip("torch")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    cache = wush.kv4_cache("mxfp4", 4, 2, 16, 64, device="cpu")
    assert cache.k_codes.shape == (4, 2, 16, 32) and cache.v_scales.shape == (4, 2, 16, 2)
    slots, ids = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        wush.kv4_append("mxfp4", bf(3, 2, 64), bf(3, 2, 64), cache, slots)
    with pytest.raises(TypeError, match="bfloat16"):
        wush.kv4_append("mxfp4", bf(3, 2, 64).float(), bf(3, 2, 64), cache, slots)
    with pytest.raises(ValueError, match="contiguous rows"):
        wush.kv4_append("mxfp4", bf(3, 64, 2).transpose(1, 2), bf(3, 2, 64), cache, slots)
    with pytest.raises(ValueError, match="tokens, heads, D"):
        wush.kv4_attention("mxfp4", bf(3, 128), cache, ids.view(3, 1), ids)
    with pytest.raises(ValueError, match="fmt must be"):
        wush.kv4_cache("fp4", 1, 1, 16, 64)
    with pytest.raises(ValueError, match="device tensor"):
        wush.linear_w4_lora("mxfp4", bf(3, 64), torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8),
                            wush.LoraAdapters(bf(1, 8, 64), bf(1, 8, 8)), ids)
    with pytest.raises(TypeError, match="logits must be"):
        wush.adjust_logits(torch.zeros(2, 8, dtype=torch.float64))
    with pytest.raises(ValueError, match="contiguous rows"):
        wush.adjust_logits(torch.zeros(8, 2).t())


class _Fake:
    """Stands in for the library: takes every call."""

    def __getattr__(self, name):
        return lambda *args: 0


def test_wrappers_check_their_tensors(monkeypatch):
    torch = pytest.importorskip("torch")
    from mxfp4_activation_amd import decode, kv4

    monkeypatch.setattr(_lib, "load", lambda: _Fake())
    for m in (decode, kv4):
        monkeypatch.setattr(m, "_enter", lambda t, name: (t.device, 0))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    cache = wush.kv4_cache("int4", 4, 2, 16, 64, device="cpu")
    k, slots = bf(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    wush.kv4_append("int4", k, k, cache, slots, T_k=bf(2, 2, 32, 32))
    for bad, error in ((dict(v=bf(3, 2, 128)), "shape of k"), (dict(slots=slots[:2]), "slots"),
                       (dict(slots=slots.int()), "slots"), (dict(T_k=bf(2, 4, 32, 32)), "T_k"),
                       (dict(cache=cache._replace(v_codes=cache.v_codes[:2])), "cache.v_codes"),
                       (dict(cache=cache._replace(k_scales=cache.k_scales.view(torch.uint8))), "cache.k_scales"),
                       (dict(k=bf(3, 4, 64), v=bf(3, 4, 64)), "heads")):
        with pytest.raises((ValueError, TypeError), match=error):
            wush.kv4_append("int4", **{**dict(k=k, v=k, cache=cache, slots=slots), **bad})
    with pytest.raises(ValueError, match="cache.k_global"):
        wush.kv4_append("nvfp4", k, k, wush.kv4_cache("nvfp4", 4, 2, 16, 64, device="cpu"), slots)
    q, table = bf(5, 4, 64), i32(3, 7)
    assert wush.kv4_attention("int4", q, cache, table[:, :6], i32(3), q_start=i32(4)).shape == (5, 4, 64)
    for bad, error in ((dict(block_table=table.long()), "block_table"), (dict(block_table=table.t()), "contiguous rows"),
                       (dict(lengths=i32(2)), "lengths"), (dict(q_start=i32(3)), "q_start"), (dict(T_q=bf(1, 2, 32, 32)), "T_q"),
                       (dict(out=bf(5, 4, 128)), "out"), (dict(q=bf(5, 4, 128)), "cache.k_codes")):
        with pytest.raises((ValueError, TypeError), match=error):
            wush.kv4_attention("int4", **{**dict(q=q, cache=cache, block_table=table, lengths=i32(3), q_start=i32(4)), **bad})
    codes, scales = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    lora = dict(x=bf(3, 64), codes=codes, scales=scales, adapters=wush.LoraAdapters(bf(2, 8, 64), bf(2, 8, 8)), ids=i32(3))
    assert wush.linear_w4_lora("mxfp4", **lora).shape == (3, 8)
    for bad, error in ((dict(ids=i32(2)), "ids"), (dict(adapters=wush.LoraAdapters(bf(2, 8, 64), bf(2, 8, 16))), "adapters.B"),
                       (dict(adapters=wush.LoraAdapters(bf(2, 8, 32), bf(2, 8, 8))), "adapters.A"),
                       (dict(adapters=wush.LoraAdapters(bf(2, 8, 64), bf(2, 8, 8), torch.ones(3))), "adapters.scale")):
        with pytest.raises((ValueError, TypeError), match=error):
            wush.linear_w4_lora("mxfp4", **{**lora, **bad})
    l = torch.zeros(3, 70)
    assert wush.adjust_logits(l, out=l) is l
    for bad, error in ((dict(prompt=i32(2, 5)), "prompt"), (dict(output=i32(3)), "output"), (dict(repetition=torch.ones(2)), "repetition"),
                       (dict(bias_ids=i32(3, 2)), "go together"), (dict(bias_ids=i32(3, 2), bias=torch.ones(3, 3)), "bias"),
                       (dict(allowed=i32(3, 2)), "allowed"), (dict(out=torch.zeros(3, 71)), "out")):
        with pytest.raises((ValueError, TypeError), match=error):
            wush.adjust_logits(l, **bad)


def _columns(shape, D):
    return 16 * (1 if shape == 0 or D > 128 else 2) * (4 if shape == 2 else 1)


def test_pieces_fit_their_workspace():
    """The rules by which the kernels cut items into pieces, restated, over random batches:
    all pieces have a workgroup, and those of cut items a place in the workspace."""
    lib, rng = wush.load(), random.Random(5)
    unit, run_units, join_units, alone_units = 128, 12, 6, 4
    for _ in range(400):
        B, kv, group, D, page = rng.choice((1, 3, 40, 200)), rng.choice((1, 8)), rng.choice((1, 4, 7)), 128, 16
        most = rng.choice((1, 3, 30, 500))
        counts = [rng.randint(0, most) for _ in range(B)]
        n = sum(counts)
        if n == 0:
            continue
        width = rng.choice((40, 300, 9000))
        lengths = [rng.choice((rng.randint(0, width * page), rng.randint(0, 200), width * page)) for _ in range(B)]
        window = rng.choice((0, 0, 100, 3000))
        columns = n * group // B
        shape = 0 if columns <= 16 else 1 if columns <= 64 else 2
        nc = _columns(shape, D)
        items = (n * group // nc + min(B, n)) * kv
        ws = lib.wush_kv4_attention_workspace(0, B, n, kv * group, kv, D, page, width)
        piece = 4 * nc * (D + 2)
        runs = (ws - 32 * (1 + items)) // (2 * piece)
        assert runs > 0 and ws == 32 * (1 + items) + 2 * runs * piece
        all_units = []
        for c, L in zip(counts, lengths):
            for t in range(-(-c * group // nc)):
                i0, i1 = t * nc // group, min((t * nc + nc - 1) // group, c - 1)
                hi, lo = max(0, L - c + i1 + 1), max(0, L - c + i0 - window + 1) if window else 0
                all_units += [-(-hi // unit) - lo // unit if hi > lo else 1] * kv
        assert len(all_units) <= items
        total = sum(all_units)
        meeting = 0 if shape == 2 else join_units * runs
        if max(all_units) * -(-len(all_units) // runs) * runs <= 1.1 * total + meeting:
            assert len(all_units) <= items + runs
            continue
        share = max(-(-total // runs), 1 if shape == 2 else min(alone_units, -(-total // 256)))
        if share >= run_units:
            assert share * runs >= total
            continue
        pieces = [-(-u // share) for u in all_units]
        assert sum(pieces) <= items + runs
        assert sum(p for p in pieces if p > 1) <= 2 * runs
        for u, p in zip(all_units, pieces):
            each = -(-u // p)
            assert each <= share and (p - 1) * each < u <= p * each


def test_attention_refuses_scales_past_fp32_as_powers_of_two():
    """The kernels take scale * log2 e: a finite scale whose product is not is refused."""
    lib = wush.load()

    def attend(scale):
        return lib.wush_kv4_attention(0, A, 1024, None, A * 10, A * 11, None, A * 13, A * 14, None, A * 3, 40, 40, A * 4, None,
                                      0, 0, 8, 2, 128, 16, 9, scale, 0, A * 5, A * 6, 1 << 40, None)

    assert attend(2.35e38) == OK and attend(1e-45) == OK
    assert attend(2.4e38) == EINVAL and b"scale" in lib.wush_last_error()


def test_adjust_refuses_outputs_that_its_counts_cannot_hold():
    """A token's count shares its word with two marks: 30 bits."""
    lib = wush.load()

    def adjust(n):
        return lib.wush_adjust_logits(A, 0, 50, 0, 50, None, 0, A * 3, n, None, None, None, None, None, 0, None, A * 9, 50, None)

    assert adjust((1 << 30) - 1) == OK
    assert adjust(1 << 30) == EINVAL and b"n_output" in lib.wush_last_error()
