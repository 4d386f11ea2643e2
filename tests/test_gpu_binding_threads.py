"""The native marshalling leaves Python's lock to other threads while it allocates and launches."""

import ctypes
import threading
import time

import numpy as np
import pytest

from tests.decode_cases import dev_bf16
from tests.kv4_cases import Batch
from tests.test_gpu_lora import Case as Lora

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture
def rebound():
    """f(name): the library's entry of that name becomes the C library's sleep(), whose argument
    is then the call's first one: the format, 1 for NVFP4."""
    from mxfp4_activation_amd import _lib

    native = _lib.binding()
    assert native is not None, "the native marshalling is not built"
    lib, libc = _lib.load(), ctypes.CDLL(None)
    at = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    own = {name: at(getattr(lib, name)) for name in _lib._NATIVE}
    yield lambda name: native.bind({**own, name: at(libc.sleep)})
    native.bind(own)


@pytest.mark.parametrize("entry", ["wush_dequant", "wush_kv4_append", "wush_kv4_attention", "wush_linear_w4_lora"])
def test_other_threads_run_during_a_call(rebound, entry):
    import mxfp4_activation_amd as wush

    b = Batch(np.random.default_rng(1), "nvfp4", 128, 2, 4, 16, [70, 30], [1, 1])
    cache, k = b.cache(), dev_bf16(b.q_bits)[:, :2]
    lora = Lora("nvfp4", 3, 40, 64, 8, 2).args()
    slots = torch.arange(2, device="cuda")
    rows = lambda t: t.view(-1, t.shape[-1])  # noqa: E731
    call = {
        "wush_dequant": lambda: wush.dequant("nvfp4", rows(cache.k_codes), rows(cache.k_scales), cache.k_global),
        "wush_kv4_append": lambda: wush.kv4_append("nvfp4", k, k, cache, slots),
        "wush_kv4_attention": lambda: b.run(cache),
        "wush_linear_w4_lora": lambda: wush.linear_w4_lora(**lora),
    }[entry]
    call()
    torch.cuda.synchronize()
    rebound(entry)
    turns, done = 0, False

    def other():
        nonlocal turns
        while not done:
            time.sleep(0.01)
            turns += 1

    thread = threading.Thread(target=other)
    thread.start()
    time.sleep(0.05)
    before = turns
    call()
    during = turns - before
    done = True
    thread.join()
    assert during >= 20  # of about 100 in the second that the call takes
