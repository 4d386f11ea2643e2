"""Transformed keys and values whose sums leave the fp32 range on the way and come back to it:
the cache holds what the exact sums become."""

import numpy as np
import pytest

from oracle import kv4 as ref
from tests.decode_cases import FMTS, bf16, dev, dev_bf16
from tests.kv4_cases import GROUP

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("run", [1, 2, 3, 4, 6, 12])
def test_sums_that_overflow_on_the_way(fmt, run):
    """Every fourth output adds huge channels with signs that alternate in runs, and comes to 0;
    the others take a few small channels alone."""
    import mxfp4_activation_amd as wush

    G, D, heads, n, page = GROUP[fmt], 64, 2, 40, 16
    if G == 16 and run in (4, 12):
        run = 6 if run == 12 else 1
    rng = np.random.default_rng(run)
    huge = G * 3 // 4
    x = np.zeros((n, heads, D))
    for c in range(0, D, G):
        x[:, :, c : c + huge] = 2.0**127 * rng.choice([1.0, 1.5], size=(n, heads, 1))
        x[:, :, c + huge : c + G] = rng.standard_normal((n, heads, G - huge))
    T = np.zeros((heads, D // G, G, G))
    T[..., :, huge:] = rng.standard_normal((heads, D // G, G, G - huge))
    over = np.arange(G) % 4 == 1
    T[..., over, huge:] = 0
    T[..., over, :huge] = np.where(np.arange(huge) // run % 2 == 0, 1.0, -1.0)
    (x, xb), (T, Tb) = bf16(x), bf16(T)
    assert np.all(T[..., over, :].sum(-1) == 0)
    g = np.float32(0.02) if fmt == "nvfp4" else None
    gs = None if g is None else dev(np.array([g]))
    pages = -(-n // page)
    cache = wush.kv4_cache(fmt, pages, heads, page, D, k_global=gs, v_global=gs)
    wush.kv4_append(fmt, dev_bf16(xb), dev_bf16(xb), cache, torch.arange(n, device="cuda"), T_k=dev_bf16(Tb))
    codes, scales = ref.append(x, fmt, T, g)
    at = np.arange(n)
    got_s = cache.k_scales.view(torch.int16) if fmt == "int4" else cache.k_scales
    assert np.array_equal(got_s.cpu().numpy().view(scales.dtype)[at // page, :, at % page], scales)
    assert np.array_equal(cache.k_codes.cpu().numpy()[at // page, :, at % page], codes)
