"""GPU parity of the mixture-of-experts layer (wush_moe_w4) with the float64
oracle.  Router operands are small integers, so the logits are fp32 numbers and the
choice of experts, ties included, must match exactly; outputs and weights
must lie within the oracle's bound, plus 2^-8 |y| for a bf16 result."""

import numpy as np
import pytest

from oracle import decode
from tests import decode_cases as dc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


def _inputs(fmt, M, E, H, I, transform, seed, ties=False):
    rng = np.random.default_rng(seed)
    G = decode.GROUP[fmt]
    # Multiples of 1/4 up to 4: distinct dot products with the router, mostly.
    x, xb = dc.bf16(rng.integers(-16, 17, size=(M, H)) / 4.0)
    step = 8.0 if ties else 64.0
    router, rb = dc.bf16(rng.integers(-2 if ties else -16, 3 if ties else 17, size=(E, H)) / (step * max(1, H // 256)))
    gc, gs = dc.weights(rng, fmt, (E, 2 * I), H)
    dcodes, ds = dc.weights(rng, fmt, (E, H), I)
    gg = dg = None
    if fmt == "nvfp4":
        gg, dg = ((2e-5 + 4e-5 * rng.random(E)).astype(np.float32) for _ in range(2))
    t_in = t_mid = None
    if transform:
        t_in = dc.bf16(rng.standard_normal((H // G, G, G)) / G**0.5)
        t_mid = dc.bf16(rng.standard_normal((E, I // G, G, G)) / G**0.5)
    return (x, xb), (router, rb), (gc, gs, gg, t_in), (dcodes, ds, dg, t_mid)


def _device_experts(fmt, p):
    import mxfp4_activation_amd as wush

    return wush.W4Experts(dc.dev(p[0]), dc.dev_scales(fmt, p[1]), None if p[2] is None else dc.dev(p[2]),
                          None if p[3] is None else dc.dev_bf16(p[3][1]))


def _oracle_experts(p):
    return (p[0], p[1], None if p[2] is None else p[2].astype(np.float64), None if p[3] is None else p[3][0])


def _run(fmt, x, router, gu, dn, k, renorm, out_dtype):
    import mxfp4_activation_amd as wush

    return wush.moe_w4(fmt, dc.dev_bf16(x[1]), dc.dev_bf16(router[1]), _device_experts(fmt, gu),
                       _device_experts(fmt, dn), k, renormalize=renorm, out_dtype=out_dtype)


def _check(fmt, got, x, router, gu, dn, k, renorm, out_dtype):
    planes = 3 if out_dtype == torch.float32 else 2
    y, bound, ids, w = decode.moe(x[0], router[0], _oracle_experts(gu), _oracle_experts(dn), k, renorm, fmt, planes)
    assert np.array_equal(got.ids.cpu().numpy(), ids)
    assert np.all(np.abs(dc.values(got.weights) - w) <= 2.0**-19 * w + 2.0**-126)
    if out_dtype == torch.bfloat16:
        bound = bound + 2.0**-8 * np.abs(y)
    err = np.abs(dc.values(got.out) - y)
    assert np.all(err <= bound), np.max(err / bound)


# (M, E, k, H, I): one token; fewer and more experts than a wave's 64 lanes, 128, 256;
# all experts chosen; a single expert with many tokens (wide and cut tiles); a
# second chunk of tokens; widths off the 128-element steps and the 32-row tiles.
_SHAPES = [(1, 4, 2, 128, 64), (1, 1, 1, 32, 32), (3, 70, 5, 160, 96), (5, 130, 8, 256, 128), (7, 300, 4, 64, 160),
           (9, 6, 6, 96, 224), (40, 2, 1, 128, 96), (64, 5, 3, 288, 64), (70, 16, 2, 128, 128), (33, 3, 2, 64, 32),
           (64, 1, 1, 64, 64)]


@pytest.mark.parametrize("transform", [False, True])
@pytest.mark.parametrize("M,E,k,H,I", _SHAPES)
@pytest.mark.parametrize("fmt", dc.FMTS)
def test_parity(fmt, M, E, k, H, I, transform):
    if fmt == "nvfp4" and I % 64 == 32:
        I += 16  # half a 32-row tile, half a group of 32
    args = _inputs(fmt, M, E, H, I, transform, 100 + M + E)
    for renorm, dt in ((True, torch.bfloat16), (False, torch.float32)):
        got = _run(fmt, *args, k, renorm, dt)
        _check(fmt, got, *args, k, renorm, dt)


def test_ties_go_to_the_lower_expert():
    args = _inputs("mxfp4", 16, 100, 32, 32, False, 5, ties=True)
    logits = args[0][0] @ args[1][0].T
    assert any(len(np.unique(r)) < 100 for r in logits)
    _check("mxfp4", _run("mxfp4", *args, 8, True, torch.float32), *args, 8, True, torch.float32)


def test_equal_logits():
    x, router, gu, dn = _inputs("int4", 4, 9, 64, 32, False, 6)
    router = (np.zeros_like(router[0]), np.zeros_like(router[1]))
    got = _run("int4", x, router, gu, dn, 3, False, torch.float32)
    assert got.ids.cpu().tolist() == [[0, 1, 2]] * 4
    _check("int4", got, x, router, gu, dn, 3, False, torch.float32)


def test_repeats_bit_for_bit():
    args = _inputs("nvfp4", 64, 24, 256, 192, True, 8)
    first = _run("nvfp4", *args, 6, True, torch.float32)
    for _ in range(3):
        again = _run("nvfp4", *args, 6, True, torch.float32)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_nan_token_stays_its_own():
    """A NaN token gives NaN, valid ids, and leaves the other tokens alone."""
    x, router, gu, dn = _inputs("mxfp4", 5, 12, 128, 64, False, 9)
    clean = _run("mxfp4", x, router, gu, dn, 3, True, torch.float32)
    xb = x[1].copy()
    xb[2, 7] = 0x7FC0
    got = _run("mxfp4", (x[0], xb), router, gu, dn, 3, True, torch.float32)
    ids = got.ids.cpu().numpy()
    assert ids.min() >= 0 and ids.max() < 12 and len(set(ids[2])) == 3
    assert torch.isnan(got.out[2]).all()
    keep = [0, 1, 3, 4]
    assert np.array_equal(ids[keep], clean.ids.cpu().numpy()[keep])
    a, b = dc.values(got.out)[keep], dc.values(clean.out)[keep]
    assert np.allclose(a, b, rtol=0, atol=1e-4 * np.abs(b).max())


def test_graph_replay_and_empty():
    import mxfp4_activation_amd as wush

    fmt = "mxfp4"
    sets = [_inputs(fmt, 6, 20, 128, 64, True, s) for s in (1, 2, 3)]
    _, router, gu, dn = sets[0]
    dgu, ddn, drouter = _device_experts(fmt, gu), _device_experts(fmt, dn), dc.dev_bf16(router[1])
    xs = [dc.dev_bf16(s[0][1]) for s in sets]
    eager = [wush.moe_w4(fmt, x, drouter, dgu, ddn, 4) for x in xs]
    torch.cuda.synchronize()
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = wush.moe_w4(fmt, x, drouter, dgu, ddn, 4)
    for turn in (0, 1, 2, 0):
        x.copy_(xs[turn])
        graph.replay()
        for a, b in zip(got, eager[turn]):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
    none = wush.moe_w4(fmt, xs[0][:0], drouter, dgu, ddn, 4)
    assert none.out.shape == (0, 128) and none.ids.shape == (0, 4)
