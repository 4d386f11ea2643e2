"""The native marshalling of the wrappers against the one in Python: the same results and
the same refusals."""

import numpy as np
import pytest

from tests.decode_cases import dev, dev_bf16
from tests.kv4_cases import Batch
from tests.test_gpu_adjust_logits import Case as Logits
from tests.test_gpu_lora import Case as Lora

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


class _Watched:
    """The native module, noting what it leaves to Python."""

    def __init__(self, module):
        self.module, self.left = module, []

    def __getattr__(self, name):
        def call(*args):
            r = getattr(self.module, name)(*args)
            if r is None:
                self.left.append(name)
            return r
        return call


@pytest.fixture
def both(monkeypatch):
    """f -> (f() natively, f() in Python); natively nothing may be left over."""
    from mxfp4_activation_amd import _lib

    native = _lib.binding()
    assert native is not None, "the native marshalling is not built"

    def run(f):
        watched = _Watched(native)
        monkeypatch.setattr(_lib, "binding", lambda: watched)
        a = f()
        assert not watched.left
        monkeypatch.setattr(_lib, "binding", lambda: None)
        return a, f()
    return run


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "int4"])
@pytest.mark.parametrize("T", [False, True])
def test_same_results(both, fmt, T):
    import mxfp4_activation_amd as wush

    b = Batch(np.random.default_rng(1), fmt, 128, 2, 4, 16, [700, 30], [3, 2], T=T)
    cache = b.cache()
    x, y = both(lambda: b.run(cache, window=50))
    assert torch.equal(x, y)
    out = torch.empty_like(x)
    x, y = both(lambda: b.run(cache, out=out, scale=0.05))
    assert x is out and y is out
    one = Batch(np.random.default_rng(2), fmt, 64, 1, 2, 32, [50, 60, 70], [1, 1, 1], T=T)
    x, y = both(lambda: wush.kv4_attention(fmt, dev_bf16(one.q_bits), one.cache(), dev(one.table), dev(one.lengths),
                                           T_q=None if not T else dev_bf16(one.T_bits)))
    assert torch.equal(x, y)
    k = dev_bf16(b.q_bits)[:, :2]
    bank = None if not T else dev_bf16(b.T_bits)

    def append():
        c = b.cache()
        wush.kv4_append(fmt, k, k, c, torch.arange(len(k), device="cuda") * 3, T_k=bank)
        return c

    for p, q in zip(*both(append)):
        assert p is None or torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    rows = lambda t: t.view(-1, t.shape[-1])  # noqa: E731
    x, y = both(lambda: wush.dequant(fmt, rows(cache.k_codes), rows(cache.k_scales), cache.k_global))
    assert x.dtype == torch.float32 and x.shape[1] == 128 and torch.equal(x, y)
    x, y = both(lambda: wush.dequant(fmt, rows(cache.v_codes), rows(cache.v_scales), cache.v_global, out=y))
    assert x is y
    lora = Lora(fmt, 12, 100, 256, 16, 3, T=T).args()
    for dtype in (torch.bfloat16, torch.float32):
        x, y = both(lambda: wush.linear_w4_lora(**lora, out_dtype=dtype))
        assert x.dtype == dtype and torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_same_logits(both, dtype):
    import mxfp4_activation_amd as wush

    c = Logits(3, 777, dtype, 9, 8, 7, True, pad=3)
    x, y = both(lambda: wush.adjust_logits(c.logits, **c.kwargs()))
    assert x.dtype == c.dtype and torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    x, y = both(lambda: wush.adjust_logits(c.logits))
    assert torch.equal(x, c.logits) and torch.equal(y, c.logits)
    l = c.logits.clone()
    x, _ = both(lambda: wush.adjust_logits(l, out=l))
    assert x is l


def test_same_refusals():
    """What is wrong on the device raises what it raises in Python, and the library's own
    refusals come through."""
    import mxfp4_activation_amd as wush

    b = Batch(np.random.default_rng(1), "mxfp4", 128, 2, 4, 16, [70, 30], [1, 1])
    cache, q, table, lengths = b.cache(), dev_bf16(b.q_bits), dev(b.table), dev(b.lengths)
    for bad, error in ((dict(lengths=lengths.cpu()), "lengths"), (dict(q=q.float()), "bfloat16"), (dict(q=q[:1]), "q_start|one query"),
                       (dict(cache=cache._replace(v_scales=cache.v_scales[1:])), "cache.v_scales"),
                       (dict(window=-1), "window"), (dict(scale=-1.0), "scale"), (dict(out=q[:, :4]), "out"), (dict(fmt="fp8"), "fmt")):
        with pytest.raises((ValueError, TypeError, wush.WushError), match=error):
            wush.kv4_attention(**{**dict(fmt="mxfp4", q=q, cache=cache, block_table=table, lengths=lengths), **bad})
    with pytest.raises(wush.WushError, match="overlap"):
        wush.kv4_attention("mxfp4", q, cache, table, lengths, out=q)
    with pytest.raises(ValueError, match="k has"):
        wush.kv4_append("mxfp4", q, q, cache, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(wush.WushError, match="page"):
        wush.kv4_append("mxfp4", q[:, :2], q[:, :2], wush.kv4_cache("mxfp4", 4, 2, 24, 128),
                        torch.zeros(2, dtype=torch.int64, device="cuda"))
    codes, scales = (t.view(-1, t.shape[-1]) for t in cache[:2])
    for bad in (dict(scales=scales[1:]), dict(codes=codes[:, ::2]), dict(out=torch.empty(1, 128, device="cuda")), dict(fmt="nvfp4")):
        with pytest.raises(ValueError, match="contiguous|shape|global_scale"):
            wush.dequant(**{**dict(fmt="mxfp4", codes=codes, scales=scales), **bad})
    a = Lora("nvfp4", 3, 40, 64, 8, 2).args()
    with pytest.raises(ValueError, match="global_scale"):
        wush.linear_w4_lora(**{**a, "global_scale": None})
    with pytest.raises(wush.WushError, match="rank"):
        wush.linear_w4_lora(**{**a, "adapters": wush.LoraAdapters(a["adapters"].A[:, :4].contiguous(), a["adapters"].B[..., :4].contiguous())})
    with pytest.raises(ValueError, match="go together"):
        wush.adjust_logits(torch.zeros(2, 9, device="cuda"), bias=torch.zeros(2, 1, device="cuda"))
    with pytest.raises(wush.WushError, match="overlap"):
        l = torch.zeros(3, 9, device="cuda")
        wush.adjust_logits(l[:2], out=l[1:])
