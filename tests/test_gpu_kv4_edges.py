"""Attention over the 4-bit cache where it can go wrong: single tokens that outweigh all
others, lengths and pages out of range, places that nothing wrote, batches of any
make, captured graphs, other streams, caches beyond 4 GiB."""

import numpy as np
import pytest

from oracle import kv4 as ref
from oracle.decode import weights as weight_values
from tests.decode_cases import FMTS, bf16, dev, dev_bf16, dev_scales, values
from tests.kv4_cases import GROUP, Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("count", [1, 9, 70])
def test_one_token_outweighs_all(fmt, D, count):
    """Every place in turn holds the one key that matters: the result is its value."""
    rng = np.random.default_rng(D + count)
    L = [300, 131, 1000, 64, 17 + count]
    b = Batch(rng, fmt, D, 2, 2, 16, L, [min(count, x) for x in L])
    one = {"mxfp4": 0x22, "nvfp4": 0x22, "int4": 0x11}[fmt]  # codes of 1.0
    b.k[0][:] = 0
    b.k[1][:] = {"mxfp4": 127, "nvfp4": 56, "int4": 0x3C00}[fmt]  # scales of 1.0
    if fmt == "nvfp4":
        b.g = (np.float32(1.0), b.g[1])
    b.q, b.q_bits = bf16(np.full_like(b.q, 512.0 / D**0.5))  # score of the one key: 512
    want = np.zeros_like(b.q)
    for s, n in enumerate(b.lengths):
        # (the first query sees it as well)
        at = int(rng.integers(0, n - b.counts[s] + 1))
        page, place = b.table[s, at // b.page], at % b.page
        b.k[0][page, :, place] = one
        v = weight_values(b.v[0][page, :, place], b.v[1][page, :, place], fmt, b.g[1])
        if fmt == "int4":  # up to 14 bits: values enter the sums with fp16's 11, then the result has 8
            v = (v / 8).astype(np.float16).astype(np.float64) * 8
        want[b.start[s] : b.start[s + 1]] = np.repeat(v, b.group, 0)
    got = b.run().double().cpu().numpy()
    assert np.array_equal(got, bf16(want)[0])


def _random_batch(rng, fmt, **kw):
    D = int(rng.choice([64, 128, 256]))
    B = int(rng.choice([1, 2, 5, 40]))
    most = int(rng.choice([1, 1, 4, 60]))
    lengths = [int(rng.integers(0, int(rng.choice([20, 400, 1500])))) for _ in range(B)]
    counts = [int(rng.integers(0, most + 1)) for _ in range(B)]
    counts[int(rng.integers(0, B))] = most
    return Batch(rng, fmt, D, int(rng.choice([1, 2, 3])), int(rng.choice([1, 3, 4, 8])), int(rng.choice([16, 64, 256])), lengths,
                 counts, T=bool(rng.random() < 0.3), **kw)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("seed", range(12))
def test_any_batch(fmt, seed):
    """Sequences without tokens, without queries, with more queries than tokens (their first
    ones see nothing), in any mixture; windows of any width."""
    rng = np.random.default_rng(seed)
    b = _random_batch(rng, fmt)
    b.check(window=int(rng.choice([0, 0, 5, 200])))


@pytest.mark.parametrize("B", [64, 65, 300, 520])
def test_many_sequences(B):
    rng = np.random.default_rng(B)
    lengths = rng.integers(0, 90, size=B)
    lengths[B // 2] = 2500
    Batch(rng, "mxfp4", 64, 2, 2, 16, lengths, rng.integers(0, 3, size=B), width=160).check()


def test_an_equal_batch_is_not_cut():
    rng = np.random.default_rng(1)
    b = Batch(rng, "int4", 128, 8, 1, 64, [900] * 96, [1] * 96)  # one piece per head and sequence
    b.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [40, 33, 64, 50]])
def test_lengths_and_pages_out_of_range(fmt, counts):
    rng = np.random.default_rng(7)
    b = Batch(rng, fmt, 128, 2, 4, 16, [300, 800, 64, 700], counts)
    good = b.run()
    for change in ("page", "negative page", "length", "negative length"):
        table, lengths = b.table.copy(), b.lengths.copy()
        if change == "page":
            table[1, 20] = b.pages
        elif change == "negative page":
            table[1, 20] = -1
        elif change == "length":
            lengths[1] = b.table.shape[1] * b.page + 1
        else:
            lengths[1] = -5
        import mxfp4_activation_amd as wush

        got = wush.kv4_attention(fmt, dev_bf16(b.q_bits), b.cache(), dev(table), dev(lengths), q_start=dev(b.start))
        lo, hi = b.start[1], b.start[2]
        if change == "negative length":
            assert torch.all(got[lo:hi] == 0)
        else:
            assert torch.isnan(got[lo:hi]).all()
        # The others: the same up to where their items are cut.
        others = torch.cat([got[:lo], got[hi:]]).float() - torch.cat([good[:lo], good[hi:]]).float()
        assert float(others.abs().max()) <= 2.0**-6 * float(good.float().abs().max())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[1, 1, 1], [50, 7, 90]])
@pytest.mark.parametrize("window", [0, 60])
def test_what_nothing_wrote_does_not_count(fmt, counts, window):
    """All places but the tokens that a query sees hold codes and scales of no number."""
    rng = np.random.default_rng(9)
    b = Batch(rng, fmt, 64, 2, 2, 32, [333, 20, 1100], counts)
    want, bound = b.want(window)
    nothing = {"mxfp4": 0xFF, "nvfp4": 0x7F, "int4": 0x7E00}[fmt]
    for c, s in (b.k, b.v):
        keep = np.zeros((b.pages, b.page), bool)
        for n, L in enumerate(b.lengths):
            t = np.arange(max(0, L - b.counts[n] - window + 1) if window else 0, L)
            keep[b.table[n, t // b.page], t % b.page] = True
        s.transpose(0, 2, 1, 3)[~keep] = nothing
        c.transpose(0, 2, 1, 3)[~keep] = 0xFF
    got = values(b.run(window=window))
    assert np.all(np.abs(got - want) <= bound)


def test_rows_behind_the_last_sequence_stay():
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(3)
    for counts in ([1, 2, 1], [60, 70, 80]):
        b = Batch(rng, "nvfp4", 128, 2, 2, 16, [40, 300, 90], counts)
        q = torch.cat([dev_bf16(b.q_bits), torch.full((5, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
        out = torch.full_like(q, 7.0)
        r = wush.kv4_attention("nvfp4", q, b.cache(), dev(b.table), dev(b.lengths), q_start=dev(b.start), out=out)
        assert r is out and torch.all(out[b.n :] == 7) and torch.isfinite(out[: b.n]).all()
        want, bound = b.want()
        assert np.all(np.abs(values(out[: b.n]) - want) <= bound)
    # No sequences, no queries.
    c = b.cache()
    none = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    assert wush.kv4_attention("nvfp4", none, c, i32(0, 4), i32(0)).shape == (0, 4, 128)
    out = torch.full_like(q, 3.0)
    wush.kv4_attention("nvfp4", q, c, i32(0, 4), i32(0), q_start=i32(1), out=out)
    wush.kv4_attention("nvfp4", q, c, i32(2, 4), i32(2), q_start=i32(3), out=out)
    assert torch.all(out == 3)


def test_strides_and_scale():
    """Queries inside a wider tensor, a table inside a wider one, another scale."""
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(11)
    b = Batch(rng, "mxfp4", 128, 2, 3, 16, [90, 400], [1, 1])
    wide = torch.full((2, 11, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8] = dev_bf16(b.q_bits)
    table = torch.full((2, 77), -9, dtype=torch.int32, device="cuda")
    table[:, 3 : 3 + b.table.shape[1]] = dev(b.table)
    b.scale = 0.031
    got = wush.kv4_attention("mxfp4", wide[:, 2:8], b.cache(), table[:, 3 : 3 + b.table.shape[1]], dev(b.lengths), scale=0.031)
    want, bound = b.want()
    assert np.all(np.abs(values(got) - want) <= bound)


@pytest.mark.parametrize("counts", [[1] * 6, [30, 2, 55, 1, 9, 80]])
def test_graph_replays_with_other_lengths(counts):
    """One captured call, replayed while the lengths, pages and queries change."""
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(21)
    width = 80
    batches = [Batch(rng, "mxfp4", 128, 2, 4, 16, np.maximum(rng.integers(1, 16 * width, size=6), counts), counts, width=width)
               for _ in range(4)]
    most = max(b.pages for b in batches)
    for b in batches:
        pad = lambda a: np.concatenate([a, np.zeros((most - b.pages, *a.shape[1:]), a.dtype)])  # noqa: E731
        b.k, b.v = tuple(map(pad, b.k)), tuple(map(pad, b.v))
    first = batches[0]
    cache, q, table, lengths, start = first.cache(), dev_bf16(first.q_bits), dev(first.table), dev(first.lengths), dev(first.start)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    call = lambda: wush.kv4_attention("mxfp4", q, cache, table, lengths, q_start=start, out=out)  # noqa: E731
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for again in range(2):
        for b in batches:
            for to, what in zip((*cache[:4], q, table, lengths), (*b.cache()[:4], dev_bf16(b.q_bits), dev(b.table), dev(b.lengths))):
                to.copy_(what)
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            replayed = out.clone()
            want, bound = b.want()
            assert np.all(np.abs(values(replayed) - want) <= bound)
            assert torch.equal(call().clone(), replayed)  # bit for bit


def test_two_streams_at_once():
    rng = np.random.default_rng(31)
    a = Batch(rng, "int4", 128, 2, 4, 16, [3000, 200, 900], [1, 1, 1])
    b = Batch(rng, "nvfp4", 64, 2, 2, 16, [700, 900], [50, 60])
    ca, cb = a.cache(), b.cache()
    wa, wb = a.run(ca), b.run(cb)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        with torch.cuda.stream(s):
            got.append((a.run(ca), wa))
        with torch.cuda.stream(t):
            got.append((b.run(cb), wb))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_then_attend_beyond_4_gib(fmt):
    """Pages past 4 GiB of codes: written by kv4_append, read by kv4_attention."""
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(41)
    heads, page, D, L = 8, 256, 128, 700
    pages = (5 << 30) // (heads * page * D // 2)
    g = torch.full((1,), 0.002, device="cuda") if fmt == "nvfp4" else None
    cache = wush.kv4_cache(fmt, pages, heads, page, D, k_global=g, v_global=g)
    used = np.array([pages - 1, 5, pages - 2], np.int32)
    k, kb = bf16(rng.standard_normal((L, heads, D)))
    v, vb = bf16(rng.standard_normal((L, heads, D)))
    t = np.arange(L)
    slots = used[t // page].astype(np.int64) * page + t % page
    order = rng.permutation(L)
    wush.kv4_append(fmt, dev_bf16(kb[order]), dev_bf16(vb[order]), cache, dev(slots[order]))
    q, qb = bf16(rng.standard_normal((3, heads * 2, D)))
    got = values(wush.kv4_attention(fmt, dev_bf16(qb), cache, dev(used[None]), dev(np.array([L], np.int32)),
                                    q_start=dev(np.array([0, 3], np.int32))))
    gn = None if g is None else np.float32(0.002)
    kc, vc = ref.append(k, fmt, None, gn), ref.append(v, fmt, None, gn)
    for h in range(heads):
        m = q[:, 2 * h : 2 * h + 2].reshape(-1, D)
        part = lambda c: tuple(a[:, h].view(np.uint16) if a.dtype == np.float16 else a[:, h] for a in c)  # noqa: E731
        want, bound = ref.attention(m, part(kc), part(vc), fmt, np.repeat(L - 3 + np.arange(3), 2), D**-0.5, kg=gn, vg=gn)
        assert np.all(np.abs(got[:, 2 * h : 2 * h + 2].reshape(-1, D) - want) <= bound)


@pytest.mark.parametrize("fmt", FMTS)
def test_transformed_keys_with_transformed_queries(fmt):
    """Hadamard blocks (their own inverse) on keys, queries and values, through append and
    attention, against the definition of both."""
    import mxfp4_activation_amd as wush
    from mxfp4_activation_amd import transforms

    rng = np.random.default_rng(51)
    G, D, heads, L, page = GROUP[fmt], 128, 2, 200, 32
    bank = transforms.hadamard_bank(D // G, G, torch.device("cuda")).repeat(heads, 1, 1, 1)
    H = bank.double().cpu().numpy()
    gn = np.float32(0.003) if fmt == "nvfp4" else None
    g = None if gn is None else torch.full((1,), 0.003, device="cuda")
    (k, kb), (v, vb), (q, qb) = (bf16(rng.standard_normal((n, heads, D)) * np.where(np.arange(D) == 5, 20, 1)) for n in (L, L, 1))
    cache = wush.kv4_cache(fmt, 8, heads, page, D, k_global=g, v_global=g)
    wush.kv4_append(fmt, dev_bf16(kb), dev_bf16(vb), cache, torch.arange(L, device="cuda"), T_k=bank, T_v=bank)
    out = values(wush.kv4_attention(fmt, dev_bf16(qb), cache, torch.arange(8, dtype=torch.int32, device="cuda")[None],
                                    torch.tensor([L], dtype=torch.int32, device="cuda"), T_q=bank))
    kc, vc = ref.append(k, fmt, H, gn), ref.append(v, fmt, H, gn)
    for h in range(heads):
        part = lambda c: tuple(a[:, h] for a in c)  # noqa: E731
        want, bound = ref.attention(q[:, h], part(kc), part(vc), fmt, np.array([L - 1]), D**-0.5, T=H[h], kg=gn, vg=gn)
        assert np.all(np.abs(out[:, h] - want) <= bound)


def test_int4_scales_half_way():
    """Largest values a with a / 7 half way between two fp16 numbers: the scale is the even one."""
    import mxfp4_activation_amd as wush

    half = np.arange(2049, 4096, 2).astype(np.float64)  # 12 bits, the last one set
    n, D, page = half.size, 64, 16
    a = 7 * half * 2.0**-11
    top = bf16(a)[0]
    assert np.all(a == top + bf16(a - top)[0])
    # A transform that adds two channels forms them without an error.
    x = np.zeros((n, 1, D))
    x[:, 0, 3], x[:, 0, 5] = top, a - top
    x[:, 0, 40], x[:, 0, 41] = -top, top - a
    T = np.zeros((1, 2, 32, 32))
    T[0, 0, 7, [3, 5]] = T[0, 1, 9, [8, 9]] = 1
    T[0, 0, 1, 3] = T[0, 1, 30, 9] = 0.25
    (x, xb), (T, Tb) = bf16(x), bf16(T)
    lead = (-(-n // page), 1, page)
    cache = wush.KV4Cache(*(dev(np.zeros((*lead, D // 2), np.uint8)) if i % 2 == 0 else
                            dev_scales("int4", np.zeros((*lead, D // 32), np.uint16)) for i in range(4)))
    wush.kv4_append("int4", dev_bf16(xb), dev_bf16(xb), cache, dev(np.arange(n)), T_k=dev_bf16(Tb), T_v=dev_bf16(Tb))
    codes, scales = ref.append(x, "int4", T)
    assert np.all(scales % 2 == 0) and np.all(scales > 0)
    for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        assert np.array_equal(s.view(torch.int16).cpu().numpy().view(np.uint16).reshape(n, 1, 2), scales)
        assert np.array_equal(c.cpu().numpy().reshape(n, 1, D // 2), codes)


@pytest.mark.parametrize("lo,hi", [(0, 0x7C00), (0x7B00, 0x7C00), (1, 0x400), (0x400, 0x800)])
@pytest.mark.parametrize("count", [1, 40])
def test_int4_value_scales_of_every_size(lo, hi, count):
    """The largest fp16 scales stay finite, the smallest ones keep what their own rounding leaves."""
    rng = np.random.default_rng(hi + count)
    b = Batch(rng, "int4", 128, 2, 4, 32, [200, count + 3], [count, count])
    b.v[1][:] = rng.integers(lo, hi, size=b.v[1].shape)
    got = b.check()
    assert np.all(np.isfinite(got))


def test_more_items_to_join_than_join_at_once():
    """1120 items of 12 units by runs of 14: most of them are in two pieces."""
    rng = np.random.default_rng(77)
    lengths = rng.integers(1420, 1537, size=140)
    Batch(rng, "mxfp4", 64, 8, 1, 16, lengths, [1] * 140).check()


@pytest.mark.parametrize("fmt", FMTS)
def test_many_sequences_of_every_length(fmt):
    """More sequences than a wave has lanes, some without tokens or queries, a few cut into pieces."""
    rng = np.random.default_rng(101)
    lengths = np.where(rng.random(300) < 0.1, rng.integers(1000, 9000, size=300), rng.integers(0, 300, size=300))
    counts = rng.integers(0, 4, size=300)
    Batch(rng, fmt, 64, 2, 2, 32, lengths, counts).check()
    Batch(rng, fmt, 128, 1, 4, 16, lengths[:70], np.where(counts[:70] == 3, 40, counts[:70])).check(window=700)
