"""Registers of the cache's, attention's, adapters' and logits' kernels, from what the compiler
notes in the built library (CPU)."""

import re

import pytest

from tests import device_code

pytestmark = pytest.mark.skipif(device_code.objdump() is None, reason="llvm tools not available")

_KERNELS = ("kv4_append_kernel", "kv4_attention_kernel", "kv4_join_kernel", "lora_kernel", "lora_expand_kernel", "adjust_kernel")


def _notes(kernel):
    found = {name: n for name, n in device_code.metadata().items() if kernel in name}
    assert found, kernel
    return found


@pytest.mark.parametrize("kernel", _KERNELS)
def test_kernels_do_not_spill(kernel):
    """Attention over INT4 keys and values for two tiles of 128 channels, or 256, is known to, by
    a few registers outside its loops' operands."""
    for name, n in _notes(kernel).items():
        m = re.search(r"kv4_attention_kernelILi(\d+)ELi(\d+)ELi(\d+)E", name)
        known = m and m[1] == "2" and (m[2] == "256" or (m[2] == "128" and m[3] != "0"))
        assert n["vgpr_spill_count"] <= (40 if known else 0), (name, n)
        assert n["private_segment_fixed_size"] <= (128 if known else 0), (name, n)


def test_attention_keeps_its_workgroups():
    """Registers leave room for the workgroups that the plan counts on: waves per SIMD are 512
    registers through a wave's, in steps of 8."""
    for name, n in _notes("kv4_attention_kernel").items():
        fmt, D, shape = map(int, re.search(r"kv4_attention_kernelILi(\d+)ELi(\d+)ELi(\d+)E", name).groups())
        if shape == 0 and D <= 128:
            want = (2 if fmt == 2 else 3) if D == 128 else (3 if fmt == 2 else 4)
        else:
            want = 3 if shape == 1 and D == 64 and fmt != 2 else 2
        assert 512 // (-(-n["vgpr_count"] // 8) * 8) >= want, (name, n)


def test_products_without_adapters_have_kernels_of_their_own():
    """What adapters need of registers is not taken from linear layers without them."""
    found = {name: n["vgpr_count"] for name, n in _notes("linear_kernel").items()}
    plain = [name for name in found if name.endswith("ELb0EEEvNS_10LinearArgsE")]
    assert plain and len(plain) * 2 == len(found)
    for name in plain:
        assert found[name] <= found[name.replace("ELb0EEEvNS", "ELb1EEEvNS")], name
