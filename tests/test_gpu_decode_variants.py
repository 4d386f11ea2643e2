"""GPU parity of the decode operators' variants by tokens, experts, rows and types that
their other tests do not reach, against the float64 oracle and its bounds."""

import numpy as np
import pytest

from tests import decode_cases as dc
from tests.test_gpu_logprobs import _check as check_logprobs
from tests.test_gpu_logprobs import _typed
from tests.test_gpu_moe_w4 import _check, _device_experts, _inputs, _run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


# The choice of experts by one, two and four tokens per wave, two, four and sixteen
# experts per lane.
@pytest.mark.parametrize("M,E,k", [(16, 100, 3), (17, 100, 3), (32, 128, 8), (33, 128, 2), (20, 200, 4), (32, 129, 32),
                                   (50, 256, 5), (64, 250, 32), (20, 257, 3), (64, 1024, 2)])
def test_choice(M, E, k):
    args = _inputs("mxfp4", M, E, 64, 32, False, M + E)
    for renorm in (True, False):
        _check("mxfp4", _run("mxfp4", *args, k, renorm, torch.float32), *args, k, renorm, torch.float32)


@pytest.mark.parametrize("M", [20, 50])
@pytest.mark.parametrize("E", [100, 200])
def test_choice_of_ties(M, E):
    args = _inputs("int4", M, E, 32, 32, False, M, ties=True)
    _check("int4", _run("int4", *args, 6, True, torch.float32), *args, 6, True, torch.float32)


@pytest.mark.parametrize("which", ["in", "mid"])
@pytest.mark.parametrize("fmt", dc.FMTS)
def test_one_transform(fmt, which):
    x, router, gu, dn = _inputs(fmt, 5, 6, 160, 96, True, 3)
    if which == "in":
        dn = dn[:3] + (None,)
    else:
        gu = gu[:3] + (None,)
    for dt in (torch.bfloat16, torch.float32):
        _check(fmt, _run(fmt, x, router, gu, dn, 2, True, dt), x, router, gu, dn, 2, True, dt)


def test_row_stride_and_out_of_a_mixture():
    import mxfp4_activation_amd as wush

    x, router, gu, dn = _inputs("mxfp4", 70, 6, 160, 96, True, 4)
    want = _run("mxfp4", x, router, gu, dn, 2, True, torch.float32)
    wide = dc.dev_bf16(np.pad(x[1], ((0, 0), (8, 24))))[:, 8:168]
    out = torch.full((72, 160), 7.0, device="cuda")
    got = wush.moe_w4("mxfp4", wide, dc.dev_bf16(router[1]), _device_experts("mxfp4", gu), _device_experts("mxfp4", dn), 2,
                      out_dtype=torch.float32, out=out[1:-1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.all(out[0] == 7.0) and torch.all(out[-1] == 7.0)


# 32 elements per thread, with one workgroup per row and with several.
@pytest.mark.parametrize("top", [0, 1, 7, 32])
@pytest.mark.parametrize("R,V", [(1100, 300), (1030, 9001), (100, 50000), (300, 20001), (513, 8200)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_wide_logprobs(dtype, R, V, top):
    rng = np.random.default_rng(R + V + top)
    l, d = _typed(rng.standard_normal((R, V)) * 3, dtype)
    check_logprobs(l, d, rng.integers(0, V, size=R), top)


@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 5)])
@pytest.mark.parametrize("R,V", [(100, 45056), (600, 8192)])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_wide_logprobs_of_any_start(dtype, R, V, pad, offset):
    rng = np.random.default_rng(pad)
    big = rng.standard_normal((R, V + pad + offset)) * 2
    l, d = _typed(big, dtype)
    d[:, :offset] = float("nan")
    d[:, offset + V :] = float("nan")
    check_logprobs(l[:, offset : offset + V], d[:, offset : offset + V], rng.integers(0, V, size=R), 5)


@pytest.mark.parametrize("R", [100, 700])
def test_wide_masks_and_ties(R):
    V = 60000 if R == 100 else 9000
    rng = np.random.default_rng(R)
    l = rng.standard_normal((R, V)) * 3
    l[0] = -np.inf
    l[1, 1:] = -np.inf
    l[2, : V - 3] = -np.inf
    l[3, rng.random(V) < 0.999] = -np.inf
    l[4] = 1.5
    l[5] = rng.integers(0, 2, V)
    l[6] = np.finfo(np.float32).min
    l[7] = np.arange(V) / 256.0
    l[8] = -np.arange(V) / 256.0
    l, d = _typed(l, "f32")
    check_logprobs(l, d, rng.integers(0, V, size=R), 32)


@pytest.mark.parametrize("M", [1, 5, 20])
def test_nan_logit_ranks_last(M):
    """An expert whose router row has a NaN: chosen only where nothing else is left, and
    without a part in the others' shares where those alone are renormalized."""
    x, router, gu, dn = _inputs("mxfp4", M, 7, 64, 32, False, 12)
    bad = router[1].copy()
    bad[3, 9] = 0x7FC0
    without = np.delete(np.arange(7), 3)
    others = tuple(a[without] for a in router)
    cut = [(p[0][without], p[1][without], None, None) for p in (gu, dn)]
    for k in (2, 6):
        got = _run("mxfp4", x, (router[0], bad), gu, dn, k, True, torch.float32)
        want = _run("mxfp4", x, others, *cut, k, True, torch.float32)
        assert np.array_equal(got.ids.cpu().numpy(), without[want.ids.cpu().numpy()])
        assert torch.equal(got.weights, want.weights)
        assert torch.allclose(got.out, want.out, rtol=0, atol=2.0**-16 * float(want.out.abs().max()))
        assert torch.isnan(_run("mxfp4", x, (router[0], bad), gu, dn, k, False, torch.float32).out).all()
    got = _run("mxfp4", x, (router[0], bad), gu, dn, 7, True, torch.float32)
    assert torch.all(got.ids[:, 6] == 3) and torch.isnan(got.out).all()
