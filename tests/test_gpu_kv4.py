"""The 4-bit key/value cache and attention over it on the GPU, against float64."""

import numpy as np
import pytest

from oracle import kv4 as ref
from tests.decode_cases import FMTS, bf16, dev, dev_bf16, dev_scales
from tests.kv4_cases import GROUP, Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


# ---------------------------------------------------------------- append

def _append_case(rng, fmt, n, heads, D, page, T):
    G = GROUP[fmt]
    x = [rng.standard_normal((n, heads, D)) * 2.0 ** rng.integers(-6, 7, size=(n, heads, 1)) for _ in range(2)]
    for a in x:
        a[:, :, rng.integers(0, D)] *= 30
        a[rng.random(a.shape[:2]) < 0.1] = 0.0
    banks = [bf16(rng.standard_normal((heads, D // G, G, G)) / 4) if T else (None, None) for _ in range(2)]
    return [bf16(a) for a in x], banks


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,heads,D,page,T", [
    (1, 1, 64, 16, False), (1, 2, 128, 16, True), (5, 3, 64, 32, True), (16, 8, 128, 16, False), (17, 2, 256, 64, True),
    (333, 5, 128, 128, True), (1000, 2, 64, 256, False),
])
def test_append(fmt, n, heads, D, page, T):
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(n * 100 + D)
    (k, v), (tk, tv) = _append_case(rng, fmt, n, heads, D, page, T)
    pages = -(-n // page) + 2
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    slots[rng.random(n) < 0.15] = -1
    if n > 3:
        slots[2] = pages * page  # just outside
    g = np.float32(0.02) if fmt == "nvfp4" else None
    gs = None if g is None else dev(np.array([g]))
    codes = [rng.integers(0, 256, size=(pages, heads, page, D // 2), dtype=np.uint8) for _ in range(2)]
    scales = [rng.integers(0, 100, size=(pages, heads, page, D // GROUP[fmt])).astype(
        np.uint16 if fmt == "int4" else np.uint8) for _ in range(2)]
    cache = wush.KV4Cache(dev(codes[0]), dev_scales(fmt, scales[0]), dev(codes[1]), dev_scales(fmt, scales[1]), gs, gs)
    # Keys inside a wider tensor, as a fused projection gives them.
    wide = torch.zeros(n, heads * 2 + 1, D, dtype=torch.bfloat16, device="cuda")
    wide[:, 1 : 1 + heads] = dev_bf16(k[1])
    wush.kv4_append(fmt, wide[:, 1 : 1 + heads], dev_bf16(v[1]), cache, dev(slots),
                    T_k=None if not T else dev_bf16(tk[1]), T_v=None if not T else dev_bf16(tv[1]))
    use = (slots >= 0) & (slots < pages * page)
    for (x, _), (bank, _), c, s, got_c, got_s in zip((k, v), (tk, tv), codes, scales, (cache.k_codes, cache.v_codes),
                                                     (cache.k_scales, cache.v_scales)):
        want_c, want_s = ref.append(x, fmt, bank, g)
        c[slots[use] // page, :, slots[use] % page] = want_c[use]
        s[slots[use] // page, :, slots[use] % page] = want_s[use].astype(s.dtype)
        got = got_s.view(torch.int16) if fmt == "int4" else got_s
        assert np.array_equal(got.cpu().numpy().view(s.dtype), s)  # scales, and what no call wrote
        assert np.array_equal(got_c.cpu().numpy(), c)


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [False, True])
@pytest.mark.parametrize("lengths,counts,heads,group,page", [
    ([1], [1], 1, 1, 16),
    ([33, 1, 500, 128, 129], [1, 1, 1, 1, 1], 2, 4, 16),
    ([700, 40, 3], [3, 2, 3], 1, 8, 64),       # 24 columns
    ([300, 97], [40, 5], 2, 3, 32),            # many columns
    ([1500, 0, 31], [1, 1, 1], 3, 16, 128),    # cut into pieces, one empty
])
def test_attention(fmt, D, T, lengths, counts, heads, group, page):
    rng = np.random.default_rng(D + len(lengths))
    Batch(rng, fmt, D, heads, group, page, lengths, counts, T=T).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window", [1, 17, 130, 4000])
@pytest.mark.parametrize("counts", [[1, 1, 1], [5, 3, 2], [77, 64, 1]])
def test_window(fmt, window, counts):
    rng = np.random.default_rng(window)
    b = Batch(rng, fmt, 128, 2, 4, 32, [900, 129, 77], counts)
    # Pages that no query sees may be gone.
    for s, (L, c) in enumerate(zip(b.lengths, b.counts)):
        first = max(0, L - c - window + 1)
        b.table[s, : first // b.page] = -7
    want_table = b.table.copy()
    b.table[b.table == -7] = 0
    want, bound = b.want(window)
    b.table = want_table
    got = b.run(window=window).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= bound)
