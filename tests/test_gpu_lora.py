"""Linear layers on 4-bit weights with low-rank adapters per token on the GPU, against float64."""

import numpy as np
import pytest

from oracle import decode as ref
from oracle.decode import GROUP
from tests.decode_cases import FMTS, bf16, dev, dev_bf16, dev_scales, values, weights

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


class Case:
    def __init__(self, fmt, M, N, K, rank, E, T=False, seed=0, scaled=True):
        rng = np.random.default_rng(seed + M + N + K + rank)
        self.fmt, self.M, self.N, self.K = fmt, M, N, K
        self.codes, self.scales = weights(rng, fmt, (N,), K)
        self.g = np.float32(0.01) if fmt == "nvfp4" else None
        self.x, self.x_bits = bf16(rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 9.0, 1.0))
        G = GROUP[fmt]
        self.T, self.T_bits = bf16(rng.standard_normal((K // G, G, G)) / G**0.5) if T else (None, None)
        self.A, self.A_bits = bf16(rng.standard_normal((E, rank, K)) / K**0.5)
        self.B, self.B_bits = bf16(rng.standard_normal((E, N, rank)) / rank**0.5)
        self.s = (0.5 + rng.random(E)).astype(np.float32) if scaled else None
        self.ids = rng.integers(-1, E, size=M).astype(np.int32)

    def args(self, stride=None):
        import mxfp4_activation_amd as wush

        x = dev_bf16(self.x_bits)
        if stride:
            wide = torch.full((self.M, stride), float("nan"), dtype=torch.bfloat16, device="cuda")
            wide[:, : self.K] = x
            x = wide[:, : self.K]
        return dict(fmt=self.fmt, x=x, codes=dev(self.codes), scales=dev_scales(self.fmt, self.scales),
                    adapters=wush.LoraAdapters(dev_bf16(self.A_bits), dev_bf16(self.B_bits),
                                               None if self.s is None else dev(self.s)), ids=dev(self.ids),
                    T=None if self.T is None else dev_bf16(self.T_bits),
                    global_scale=None if self.g is None else dev(np.array([self.g])))

    def want(self, planes):
        y, b = ref.linear(self.x, self.codes, self.scales, self.fmt, self.T, self.g, planes)
        d, c = ref.lora(self.x, self.A, self.B, np.ones(len(self.A)) if self.s is None else self.s, self.ids)
        return y + d, b + c + 2 * ref.U * (np.abs(y) + np.abs(d))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,rank,E,T,out", [
    (1, 64, 256, 8, 1, False, "f32"), (1, 4096, 1024, 16, 3, False, "bf16"), (3, 77, 96, 24, 2, True, "f32"),
    (13, 500, 672, 64, 5, True, "bf16"), (33, 130, 2080, 16, 40, False, "f32"), (64, 1000, 512, 128, 7, True, "f32"),
    (70, 48, 256, 512, 2, False, "bf16"), (200, 33, 64, 8, 9, False, "f32"),
    # added in the product, and just not
    (64, 129, 256, 8, 3, False, "bf16"), (50, 300, 512, 32, 6, True, "f32"), (17, 65, 96, 24, 4, False, "f32"),
    (9, 200, 128, 40, 3, False, "bf16"), (8, 70, 128, 128, 2, True, "f32"), (8, 70, 128, 136, 2, False, "bf16"),
])
def test_lora(fmt, M, N, K, rank, E, T, out):
    import mxfp4_activation_amd as wush

    c = Case(fmt, M, N, K, rank, E, T)
    dtype = torch.float32 if out == "f32" else torch.bfloat16
    y = values(wush.linear_w4_lora(**c.args(), out_dtype=dtype))
    want, bound = c.want(3 if out == "f32" else 2)
    if out == "bf16":
        bound = bound + 2.0**-8 * (np.abs(want) + bound)
    assert np.all(np.abs(y - want) <= bound)


@pytest.mark.parametrize("fmt", FMTS)
def test_no_adapter_is_the_linear_layer(fmt):
    import mxfp4_activation_amd as wush

    c = Case(fmt, 9, 200, 256, 16, 2, T=True)
    c.ids[:] = -5
    a = c.args()
    plain = wush.linear_w4(fmt, a["x"], a["codes"], a["scales"], T=a["T"], global_scale=a["global_scale"])
    assert torch.equal(wush.linear_w4_lora(**a), plain)
    # No adapters at all.
    a["adapters"] = wush.LoraAdapters(*(t[:0].contiguous() for t in a["adapters"]))
    assert torch.equal(wush.linear_w4_lora(**a), plain)


def test_adapters_out_of_range_and_strides():
    import mxfp4_activation_amd as wush

    c = Case("mxfp4", 6, 100, 320, 16, 3, scaled=False)
    c.ids = np.array([0, 3, -1, 2, 2**31 - 1, 2], np.int32)
    y = wush.linear_w4_lora(**c.args(stride=344), out_dtype=torch.float32)
    bad = torch.isnan(y).all(1).cpu().numpy()
    assert bad.tolist() == [False, True, False, False, True, False]
    c.ids = np.where(bad, -1, c.ids).astype(np.int32)
    want, bound = c.want(3)
    assert np.all(np.abs(values(y) - want)[~bad] <= bound[~bad])
    # A token that is not finite leaves the others alone.
    a = c.args()
    a["x"][3, 5] = float("inf")
    z = wush.linear_w4_lora(**a, out_dtype=torch.float32)
    keep = [0, 1, 2, 4, 5]
    assert np.all(np.abs(values(z) - want)[keep] <= bound[keep]) and not torch.isfinite(z[3]).all()


@pytest.mark.parametrize("M", [3, 70])
def test_no_adapter_keeps_results_of_minus_zero(M):
    """A tensor scale that takes small negative sums below the fp32 range leaves -0, with
    adapters beside it as without."""
    import mxfp4_activation_amd as wush

    a = Case("nvfp4", M, 300, 64, 16, 2).args()
    a["global_scale"] = torch.full((1,), 2.0**-149, device="cuda")
    a["scales"] = torch.full_like(a["scales"], 1)  # 2^-9
    a["ids"] = torch.full_like(a["ids"], -1)
    got = wush.linear_w4_lora(**a, out_dtype=torch.float32)
    want = wush.linear_w4("nvfp4", a["x"], a["codes"], a["scales"], global_scale=a["global_scale"], out_dtype=torch.float32)
    assert torch.any((want == 0) & torch.signbit(want))
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))
