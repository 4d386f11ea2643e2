"""Attention over caches that hold values and scales that are not finite, or tensor scales of
any kind: each query's result depends on the tokens that it sees alone."""

import numpy as np
import pytest

from tests.decode_cases import FMTS, bf16, values
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
@pytest.mark.parametrize("counts", [[3, 5, 2], [12, 20, 16], [150, 70, 131]])  # 16 columns, two tiles, prompts
@pytest.mark.parametrize("window", [0, 7, 60])
def test_values_that_are_not_finite_stay_with_their_tokens(fmt, D, counts, window):
    """A token's group of values without a finite scale spoils that group's channels for the
    queries that see the token, and nothing else."""
    rng = np.random.default_rng(D + counts[0] + window)
    b = Batch(rng, fmt, D, 2, 2, 32, [333, 90, 2000], counts, T=window == 60)
    want, bound = b.want(window)
    bad = {"mxfp4": 0xFF, "nvfp4": 0x7F, "int4": 0x7C00}[fmt]
    G = GROUP[fmt]
    hit = np.zeros(want.shape, bool)
    for s, (L, c) in enumerate(zip(b.lengths, b.counts)):
        pos = np.arange(L - c, L)
        # Among the queries' own tokens, the last one among them, and one from before.
        for at in (L - c + c // 2, L - 1, L - c - 3):
            page, place, g = b.table[s, at // b.page], at % b.page, int(rng.integers(0, D // G))
            b.v[1][page, :, place, g] = bad
            b.v[0][page, :, place, g * G // 2 : (g + 1) * G // 2] = 0x77
            sees = (at <= pos) & ((window == 0) | (at > pos - window))
            rows = b.start[s] + np.nonzero(sees)[0]
            hit[rows, :, g * G : (g + 1) * G] = True
    got = values(b.run(window=window))
    assert not np.isfinite(got[hit]).any()
    assert np.all(np.abs(got - want)[~hit] <= bound[~hit])


@pytest.mark.parametrize("counts", [[3, 5, 2], [12, 20, 16], [150, 70, 131]])
def test_key_tensor_scales_of_every_kind(counts):
    """A tensor scale of 0 makes all scores 0, a tiny one counts with its own size, and one that
    is NaN or negative shows in every result."""
    rng = np.random.default_rng(counts[0])
    b = Batch(rng, "nvfp4", 128, 2, 2, 32, [333, 90, 2000], counts)
    vg = b.g[1]
    b.check()
    for bad in (np.nan, -b.g[0]):
        b.g = np.float32(bad), vg
        assert torch.isnan(b.run()).all()
    b.g = np.float32(0.0), vg
    b.check()
    # The same scores, from larger queries.
    b.g = np.float32(2e-3) * np.float32(2.0**-100), vg
    b.q, b.q_bits = bf16(b.q * 2.0**100)
    b.check()
