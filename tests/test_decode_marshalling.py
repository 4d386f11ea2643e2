"""What the decode wrappers hand to the library, with a stand-in for it that reads
host memory (no GPU needed)."""

import ctypes

import pytest

import mxfp4_activation_amd as wush

torch = pytest.importorskip("torch")


class _Library:
    """Notes the tensor scales that a call finds at the addresses it is given."""

    def __init__(self, experts):
        self.experts, self.seen = experts, []

    def _read(self, address, n):
        # An allocation of the call's own after the addresses were taken.
        torch.full((n,), -1.0)
        self.seen.append(list((ctypes.c_float * n).from_address(address)))

    def wush_linear_w4_workspace(self, *args):
        return 0

    def wush_moe_w4_workspace(self, *args):
        return 0

    def wush_linear_w4(self, fmt, x, ldx, T, codes, scales, gs, *rest):
        self._read(gs, 1)
        return 0

    def wush_moe_w4(self, fmt, x, ldx, router, gc, gs, gate_up, ti, dc, ds, down, *rest):
        self._read(gate_up, self.experts)
        self._read(down, self.experts)
        return 0


@pytest.fixture
def library(monkeypatch):
    from mxfp4_activation_amd import _lib, decode

    fake = _Library(8)
    monkeypatch.setattr(_lib, "load", lambda: fake)
    monkeypatch.setattr(decode, "_enter", lambda t, name: (t.device, 0))
    return fake


def _grid(n, first):
    """n values in a tensor that cannot be viewed flat."""
    return (torch.arange(n, dtype=torch.float32) + first).view(2, n // 2).t()


def test_moe_tensor_scales_live_until_the_call(library):
    E, H, I = 8, 32, 32
    x = torch.zeros(2, H, dtype=torch.bfloat16)
    gate, down = _grid(E, 1.0), _grid(E, 100.0)
    u8 = lambda *shape: torch.zeros(*shape, dtype=torch.uint8)  # noqa: E731
    for _ in range(20):
        library.seen.clear()
        wush.moe_w4("nvfp4", x, torch.zeros(E, H, dtype=torch.bfloat16),
                    wush.W4Experts(u8(E, 2 * I, H // 2), u8(E, 2 * I, H // 16), gate),
                    wush.W4Experts(u8(E, H, I // 2), u8(E, H, I // 16), down), 2)
        assert library.seen == [gate.reshape(-1).tolist(), down.reshape(-1).tolist()]


def test_linear_tensor_scale_of_any_one_element_shape(library):
    x, codes = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.uint8)
    for g in (torch.tensor([3.0]), torch.tensor(3.0), torch.tensor([[3.0]])):
        wush.linear_w4("nvfp4", x, codes, torch.zeros(4, 2, dtype=torch.uint8), global_scale=g)
        assert library.seen.pop() == [3.0]
