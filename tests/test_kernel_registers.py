"""Registers of the decode kernels, from what the compiler notes in the built library (CPU)."""

import pytest

from tests import device_code

pytestmark = pytest.mark.skipif(device_code.objdump() is None, reason="llvm tools not available")

_DECODE = ("linear_kernel", "split_kernel", "router_kernel", "route_kernel", "gate_up_kernel", "down_kernel",
           "combine_kernel", "logprob_kernel", "join_kernel")


def test_decode_kernels_do_not_spill():
    notes = device_code.metadata()
    mine = {name: n for name, n in notes.items() if any(k in name for k in _DECODE)}
    for kernel in _DECODE:
        assert any(kernel in name for name in mine), kernel
    spills = {name: (n["vgpr_spill_count"], n["private_segment_fixed_size"]) for name, n in mine.items()
              if n["vgpr_spill_count"] or n["private_segment_fixed_size"]}
    assert not spills, spills
