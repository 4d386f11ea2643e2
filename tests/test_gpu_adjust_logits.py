"""Penalties, biases and masks on logits on the GPU, against float64."""

import numpy as np
import pytest

from oracle import decode as ref
from tests.decode_cases import dev, values

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


class Case:
    def __init__(self, R, V, dtype, n_prompt, n_output, n_bias, masked, pad=0, seed=0):
        rng = np.random.default_rng(seed + R + V)
        self.R, self.V, self.dtype = R, V, TYPES[dtype]
        self.wide = torch.from_numpy(4 * rng.standard_normal((R, V + pad))).to(self.dtype).cuda()
        self.logits = self.wide[:, :V]
        ids = lambda n: rng.integers(-2, max(2, min(V + 2, 40)), size=(R, n)).astype(np.int32)  # noqa: E731
        self.prompt, self.output = ids(n_prompt), ids(n_output)
        for a in (self.prompt, self.output):
            a[rng.random(a.shape) < 0.3] = rng.integers(0, V)
        self.rep = (0.7 + rng.random(R)).astype(np.float32)
        self.freq, self.pres = (rng.standard_normal(R).astype(np.float32) for _ in range(2))
        self.bias_ids = rng.integers(-1, V + 1, size=(R, n_bias)).astype(np.int32)
        if n_bias > 4:
            self.bias_ids[:, 3] = self.bias_ids[:, 1]  # the same token twice and three times
            self.bias_ids[::2, 4] = self.bias_ids[::2, 1]
        self.bias = (5 * rng.standard_normal((R, n_bias))).astype(np.float32)
        self.allowed = rng.integers(0, 2**32, size=(R, (V + 31) // 32), dtype=np.uint32) if masked else None
        if masked:
            self.allowed[0] = 0

    def kwargs(self):
        part = lambda a: dev(a) if a.shape[1] else None  # noqa: E731
        return dict(prompt=part(self.prompt), output=part(self.output), repetition=dev(self.rep),
                    frequency=dev(self.freq), presence=dev(self.pres), bias_ids=part(self.bias_ids),
                    bias=part(self.bias), allowed=None if self.allowed is None else dev(self.allowed.view(np.int32)))

    def want(self):
        ok = None
        if self.allowed is not None:
            ok = np.unpackbits(self.allowed.view(np.uint8), axis=1, bitorder="little")[:, : self.V].astype(bool)
        return ref.adjust_logits(values(self.logits), self.prompt, self.output, self.rep.astype(float),
                                 self.freq.astype(float), self.pres.astype(float), self.bias_ids,
                                 self.bias.astype(float), ok)

    def check(self, got):
        want, bound = self.want()
        if self.dtype != torch.float32:
            bound = bound + torch.finfo(self.dtype).eps / 2 * (np.abs(want) + bound)
            if self.dtype == torch.float16:
                bound = bound + 2.0**-25
        gone = np.isneginf(want)
        assert np.array_equal(gone, np.isneginf(got))
        keep = ~gone
        assert np.all(np.abs(got[keep] - want[keep]) <= bound[keep])


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("R,V,n_prompt,n_output,n_bias,masked,pad", [
    (1, 1, 1, 1, 1, True, 0), (1, 1000, 5, 9, 0, False, 0), (3, 31, 0, 4, 7, True, 5), (2, 511, 17, 0, 3, False, 3),
    (5, 513, 70, 33, 300, True, 0), (7, 4097, 1025, 259, 20, True, 7), (600, 5003, 3, 2, 9, True, 1),
    (2, 140001, 2000, 999, 64, True, 0), (4, 2048, 0, 0, 0, True, 0), (4, 2050, 0, 0, 6, False, 0),
])
def test_adjust(dtype, R, V, n_prompt, n_output, n_bias, masked, pad):
    import mxfp4_activation_amd as wush

    c = Case(R, V, dtype, n_prompt, n_output, n_bias, masked, pad)
    before = c.wide.clone()
    got = wush.adjust_logits(c.logits, **c.kwargs())
    assert torch.equal(c.wide, before)
    c.check(values(got))
    # In place: the same, and nothing behind the vocabulary changes.
    again = c.wide.clone()
    view = again[:, :V]
    assert wush.adjust_logits(view, **c.kwargs(), out=view) is view
    assert torch.equal(view.contiguous().view(torch.uint8), got.view(torch.uint8))
    assert torch.equal(again[:, V:], before[:, V:])


def test_values_that_are_not_finite():
    import mxfp4_activation_amd as wush

    l = torch.zeros(2, 64, device="cuda")
    l[:, 0], l[:, 1], l[:, 2], l[:, 3] = float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min
    allowed = torch.tensor([[-1, -1], [~0xF, -1]], dtype=torch.int32, device="cuda")
    seen = torch.arange(4, dtype=torch.int32, device="cuda").repeat(2, 1)
    r = wush.adjust_logits(l, prompt=seen, repetition=torch.full((2,), 2.0, device="cuda"), allowed=allowed)
    assert torch.isnan(r[0, 0]) and r[0, 1] == float("inf") and r[0, 2] == -float("inf") and r[0, 3] == -float("inf")
    assert torch.equal(r[0, 4:], l[0, 4:])
    assert torch.isneginf(r[1, :4]).all() and torch.equal(r[1, 4:], l[1, 4:])


def test_without_anything_is_a_copy():
    import mxfp4_activation_amd as wush

    l = torch.randn(3, 1001, device="cuda").to(torch.bfloat16)
    assert torch.equal(wush.adjust_logits(l), l)
    # Penalties without lists, empty lists, padding only.
    none = torch.full((3, 5), -1, dtype=torch.int32, device="cuda")
    p = torch.full((3,), 3.0, device="cuda")
    assert torch.equal(wush.adjust_logits(l, repetition=p, frequency=p, presence=p), l)
    assert torch.equal(wush.adjust_logits(l, prompt=none, output=none[:, :0].contiguous(), repetition=p, frequency=p, presence=p), l)
    assert wush.adjust_logits(l[:0]).shape == (0, 1001)
