"""GPU parity of the 4-bit products over several chunks of K: the loop with weights
and activations in flight, the last whole chunks after it for an even and an odd
number of them, and what remains past them, for every shape of workgroup that
wush_linear_w4 and wush_moe_w4 choose from.

* Linear layers: small integers times codes with power-of-two scales, every partial
  sum an fp32 number: the result must match bit for bit, every time.
* Mixtures: within the oracle's bound, and the same bits every time.
"""

import numpy as np
import pytest

from oracle import decode
from tests import decode_cases as dc
from tests.test_gpu_moe_w4 import _check, _run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


# (M, N, chunk): tokens and weight rows that lead to a shape of workgroup, and
# the elements of K that it takes at a time.  With T there are two or three planes of
# activations (bf16 and fp32 results), which lead to others of the same list.
_SHAPES = [
    (3, 12400, 1024),  # up to four tokens, many rows
    (1, 70, 2048),     # few rows, eight waves along K
    (4, 70, 1024),     # the same, three planes: half the chunk
    (5, 70, 2048), (6, 520, 1024),
    (8, 600, 1024), (13, 600, 512),
    (8, 1100, 1024), (16, 1000, 1024),
    (16, 8200, 512),
    (20, 8300, 512), (20, 8300, 256),
    (40, 5500, 512), (64, 5500, 256),
    (24, 16500, 512), (24, 16500, 256), (40, 11000, 512),
    (50, 16500, 256), (64, 33000, 256),
]

# Whole chunks, and what remains: nothing, less than a wave's part, most waves' parts, all
# but the last group.
_PARTS = [(2, 0.6), (3, 0.3), (4, 0.05), (4, 0.0), (5, 0.0), (5, 0.3), (6, 0.99)]


@pytest.mark.parametrize("transform", [False, True])
@pytest.mark.parametrize("M,N,chunk", _SHAPES)
@pytest.mark.parametrize("fmt", dc.FMTS)
def test_linear_exact(fmt, M, N, chunk, transform):
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(1000 * M + N)
    G, some = decode.GROUP[fmt], min(N, 97)  # the rows repeat
    gs = 0.5 if fmt == "nvfp4" else None
    for whole, rest in _PARTS:
        K = whole * chunk + (max(G, int(rest * chunk) // G * G) if rest else 0)
        codes, scales = dc.weights(rng, fmt, (some,), K, exact=True)
        x, xb = dc.bf16(rng.integers(-3, 4, size=(M, K)))
        T = dT = None
        if transform:
            # Four entries of +-1 a row.
            T = np.zeros((K // G, G, G))
            at = rng.integers(0, G, size=(K // G, G, 4))
            np.put_along_axis(T, at, rng.choice([-1.0, 1.0], size=at.shape), 2)
            T, Tb = dc.bf16(T)
            dT = dc.dev_bf16(Tb)
        want = dc.dev(decode.linear(x, codes, scales, fmt, T, gs)[0])
        rows = torch.arange(N, device="cuda") % some
        args = (fmt, dc.dev_bf16(xb), dc.dev(codes)[rows].contiguous(), dc.dev_scales(fmt, scales)[rows].contiguous())
        g = None if gs is None else torch.tensor([gs], dtype=torch.float32).cuda()
        for turn in range(3):
            got = wush.linear_w4(*args, T=dT, global_scale=g, out_dtype=torch.float32)
            assert torch.equal(got.double(), want[:, rows]), (K, turn)
            got = wush.linear_w4(*args, T=dT, global_scale=g)
            assert torch.equal(got, want[:, rows].to(torch.bfloat16)), (K, turn, "bf16")


# (M, E, k): tiles of 4, 16 and 32 tokens.
_TILES = [(3, 4, 2), (16, 3, 2), (40, 3, 2)]
# Chunks of 512 or 256: three to ten, whole and not; which transforms there are.
_WIDTHS = [(1536, 1024, ""), (1696, 2080, "both"), (2048, 1568, "in"), (2592, 1312, "mid")]


def _parity_and_repeats(fmt, M, E, k, H, I, transforms):
    rng = np.random.default_rng(M + H)
    G = decode.GROUP[fmt]
    if fmt == "nvfp4":
        H, I = (w + 16 if w % 128 else w for w in (H, I))
    # Integers over a power of two: the logits are fp32 numbers.
    x = dc.bf16(rng.integers(-16, 17, size=(M, H)) / 4.0)
    router = dc.bf16(rng.integers(-16, 17, size=(E, H)) / 512.0)
    gc, gs = dc.weights(rng, fmt, (E, 2 * I), H)
    dcodes, ds = dc.weights(rng, fmt, (E, H), I)
    gg = dg = t_in = t_mid = None
    if fmt == "nvfp4":
        gg, dg = ((2e-5 + 4e-5 * rng.random(E)).astype(np.float32) for _ in range(2))
    if transforms in ("in", "both"):
        t_in = dc.bf16(rng.standard_normal((H // G, G, G)) / G**0.5)
    if transforms in ("mid", "both"):
        t_mid = dc.bf16(rng.standard_normal((E, I // G, G, G)) / G**0.5)
    args = (x, router, (gc, gs, gg, t_in), (dcodes, ds, dg, t_mid))
    for renorm, dt in ((True, torch.bfloat16), (False, torch.float32)):
        got = _run(fmt, *args, k, renorm, dt)
        _check(fmt, got, *args, k, renorm, dt)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(got, _run(fmt, *args, k, renorm, dt)))


@pytest.mark.parametrize("H,I,transforms", _WIDTHS)
@pytest.mark.parametrize("M,E,k", _TILES)
@pytest.mark.parametrize("fmt", dc.FMTS)
def test_moe(fmt, M, E, k, H, I, transforms):
    _parity_and_repeats(fmt, M, E, k, H, I, transforms)


# Tiles of 16 tokens on more experts than compute units take at a time.
@pytest.mark.parametrize("H,I,transforms", [(1024, 800, ""), (1056, 1312, "both")])
@pytest.mark.parametrize("fmt", dc.FMTS)
def test_moe_of_many_experts(fmt, H, I, transforms):
    _parity_and_repeats(fmt, 16, 40, 8, H, I, transforms)
