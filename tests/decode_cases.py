"""Seeded inputs of the decode tests, as numpy arrays and their device tensors."""

from __future__ import annotations

import numpy as np

from oracle import codecs
from oracle.decode import GROUP
from synthetic import f64_to_bf16_bits

FMTS = ["mxfp4", "nvfp4", "int4"]


def bf16(a):
    """(values after rounding to bf16 in float64, bit patterns)."""
    bits = f64_to_bf16_bits(np.asarray(a, dtype=np.float64))
    return codecs.bf16_bits_to_f32(bits).astype(np.float64), bits


def dev_bf16(bits):
    import torch

    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def dev(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_scales(fmt, scales):
    import torch

    return dev(scales.view(np.int16)).view(torch.float16) if fmt == "int4" else dev(scales)


def weights(rng, fmt, shape, K, exact=False):
    """Codes [*shape, K/2] and scales [*shape, K/G].  exact: scales are powers of
    two of a narrow range, so that sums of products with small integers are fp32
    numbers."""
    codes = rng.integers(0, 256, size=(*shape, K // 2), dtype=np.uint8)
    ss = (*shape, K // GROUP[fmt])
    if fmt == "mxfp4":
        scales = rng.integers(126, 129, size=ss, dtype=np.uint8) if exact else rng.integers(
            117, 123, size=ss, dtype=np.uint8)
    elif fmt == "nvfp4":
        # E4M3 code 8 e + m is 2^(e - 7) (1 + m / 8).
        scales = (8 * rng.integers(6, 9, size=ss)).astype(np.uint8) if exact else rng.integers(
            0, 127, size=ss, dtype=np.uint8)
    else:
        v = np.ldexp(1.0, rng.integers(-1, 2, size=ss)) if exact else 0.004 + 0.006 * rng.random(ss)
        scales = v.astype(np.float16).view(np.uint16)
    return codes, scales


def values(t):
    """A device tensor's values in float64."""
    return t.detach().double().cpu().numpy()
