"""Decoding with 4-bit weights: linear layers and mixtures of experts for a
few tokens, and the log probabilities of tokens.

The weights are what the library writes: codes and scales of the quantizers
(``quant``) or of GPTQ-WUSH, unchanged.  Like ``ops``, these functions only
marshal arguments: they allocate outputs and workspace with torch and enqueue
the library call on torch's current stream.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib

_G = {"mxfp4": 32, "nvfp4": 16, "int4": 32}
_OUT = {torch.float32: 0, torch.bfloat16: 1}
_LOGITS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


# The current stream's handle without a Stream object around it: a call on one
# token takes a few microseconds, of which building that object would be two.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _enter(t: torch.Tensor, name: str):
    """(device, raw current stream) of a call whose first operand is t."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    dev = t.device
    current = torch.cuda.current_device()
    if dev.index != current:
        raise ValueError("%s must be on the current device (it is on %s, current cuda:%d)" % (name, dev, current))
    return dev, _raw_stream(current)


def _fmt(fmt: str):
    if fmt not in _G:
        raise ValueError("fmt must be one of %s (got %r)" % (sorted(_G), fmt))
    return _lib.FMT[fmt], _G[fmt]


def _out_type(out_dtype) -> int:
    if out_dtype not in _OUT:
        raise ValueError("out_dtype must be float32 or bfloat16")
    return _OUT[out_dtype]


def _check(t, name: str, dtype, shape, dev) -> int:
    """A contiguous tensor of this dtype and shape on dev; its address."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if t.device != dev:
        raise ValueError("%s must be on %s (got %s)" % (name, dev, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows(x: torch.Tensor, name: str):
    """(rows, width, row stride) of a bf16 matrix whose rows are contiguous."""
    if x.dtype != torch.bfloat16:
        raise TypeError("%s must be bfloat16" % name)
    if x.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    M, K = x.shape
    if K > 1 and x.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    return M, K, x.stride(0)


def _scale_dtype(fmt: str):
    return torch.float16 if fmt == "int4" else torch.uint8


def _check_global(fmt: str, g, name: str, n: int, dev):
    """(address of the tensor scales, their flat tensor, which the caller holds until
    the call is enqueued: it is a copy where g cannot be viewed flat)."""
    if fmt != "nvfp4":
        return None, None
    if g is None:
        raise ValueError("nvfp4 needs %s, a float32 tensor of %d element%s" % (name, n, "" if n == 1 else "s"))
    if g.dim() != 1:
        g = g.reshape(-1)
    return _check(g, name, torch.float32, (n,), dev), g


def _workspace(n: int, dev):
    return torch.empty(n, dtype=torch.uint8, device=dev) if n else None


def linear_w4(fmt: str, x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
              T: Optional[torch.Tensor] = None, global_scale: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x' W^T for a few tokens: bf16 activations x [M, K] (rows contiguous, any
    row stride that is a multiple of 8) times the 4-bit weights codes [N, K/2],
    scales [N, K/G] (``quant`` or ``gptq_wush``), with x' = x, or the block
    transform of x by the activation bank T [K/G, G, G].  NVFP4 weights take
    their tensor scale as global_scale.  Returns [M, N] in out_dtype.  Sums are fp32;
    T x enters them with 16 significant bits where out_dtype is bfloat16 and with all
    24 where it is float32."""
    f, G = _fmt(fmt)
    ot = _out_type(out_dtype)
    M, K, ldx = _rows(x, "x")
    dev, stream = _enter(x, "x")
    if codes.dim() != 2:
        raise ValueError("codes must be 2-D")
    N = codes.shape[0]
    pc = _check(codes, "codes", torch.uint8, (N, K // 2), dev)
    ps = _check(scales, "scales", _scale_dtype(fmt), (N, K // G), dev)
    pg, global_scale = _check_global(fmt, global_scale, "global_scale", 1, dev)
    pt = None if T is None else _check(T, "T", torch.bfloat16, (K // G, G, G), dev)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
        po = out.data_ptr()
    else:
        po = _check(out, "out", out_dtype, (M, N), dev)
    lib = _lib.load()
    nw = 0 if T is None else lib.wush_linear_w4_workspace(M, K, ot)
    ws = _workspace(nw, dev)
    st = lib.wush_linear_w4(f, x.data_ptr(), ldx, pt, pc, ps, pg, M, N, K, po, ot, ws.data_ptr() if nw else None, nw,
                            stream)
    if st:
        _lib.check(st, "wush_linear_w4(%s)" % fmt)
    return out


class W4Experts(NamedTuple):
    """One projection of all experts in 4 bits: codes uint8 [E, rows, K/2],
    scales [E, rows, K/G], for NVFP4 the experts' tensor scales [E], and the block
    transforms of its input, if any."""
    codes: torch.Tensor
    scales: torch.Tensor
    global_scale: Optional[torch.Tensor] = None
    T: Optional[torch.Tensor] = None


class MoeResult(NamedTuple):
    out: torch.Tensor      # [M, H]
    ids: torch.Tensor      # int32 [M, top_k]: the chosen experts, most likely first
    weights: torch.Tensor  # float32 [M, top_k]


def moe_w4(fmt: str, x: torch.Tensor, router: torch.Tensor, gate_up: W4Experts, down: W4Experts, top_k: int,
           renormalize: bool = True, out_dtype: torch.dtype = torch.bfloat16,
           out: Optional[torch.Tensor] = None) -> MoeResult:
    """A mixture-of-experts layer for a few tokens x [M, H] (bf16): the bf16
    router [E, H], softmax over the experts, the top_k most likely ones
    (renormalized to sum 1, or not), SwiGLU experts and their weighted sum.
    gate_up holds 2 I rows per expert, I of the gate, then I of the up
    projection; its T is one bank [H/G, G, G] for all experts.  down holds H
    rows of width I; its T is [E, I/G, G, G].  Sums are fp32; the transformed x and the
    experts' inner activations enter them with 16 significant bits where out_dtype is
    bfloat16 and with all 24 where it is float32."""
    f, G = _fmt(fmt)
    ot = _out_type(out_dtype)
    M, H, ldx = _rows(x, "x")
    dev, stream = _enter(x, "x")
    if router.dim() != 2 or gate_up.codes.dim() != 3:
        raise ValueError("router must be [E, H] and gate_up.codes [E, 2 I, H/2]")
    E, rows = router.shape[0], gate_up.codes.shape[1]
    I = rows // 2
    sdt = _scale_dtype(fmt)
    pr = _check(router, "router", torch.bfloat16, (E, H), dev)
    pgc = _check(gate_up.codes, "gate_up.codes", torch.uint8, (E, 2 * I, H // 2), dev)
    pgs = _check(gate_up.scales, "gate_up.scales", sdt, (E, 2 * I, H // G), dev)
    pgg, gate_up_global = _check_global(fmt, gate_up.global_scale, "gate_up.global_scale", E, dev)
    pdc = _check(down.codes, "down.codes", torch.uint8, (E, H, I // 2), dev)
    pds = _check(down.scales, "down.scales", sdt, (E, H, I // G), dev)
    pdg, down_global = _check_global(fmt, down.global_scale, "down.global_scale", E, dev)
    pti = None if gate_up.T is None else _check(gate_up.T, "gate_up.T", torch.bfloat16, (H // G, G, G), dev)
    ptm = None if down.T is None else _check(down.T, "down.T", torch.bfloat16, (E, I // G, G, G), dev)
    if out is None:
        out = torch.empty((M, H), dtype=out_dtype, device=dev)
        po = out.data_ptr()
    else:
        po = _check(out, "out", out_dtype, (M, H), dev)
    ids = torch.empty((M, top_k), dtype=torch.int32, device=dev)
    weights = torch.empty((M, top_k), dtype=torch.float32, device=dev)
    lib = _lib.load()
    nw = lib.wush_moe_w4_workspace(M, E, top_k, H, I, 0 if pti is None else 1, ot)
    ws = _workspace(nw, dev)
    st = lib.wush_moe_w4(f, x.data_ptr(), ldx, pr, pgc, pgs, pgg, pti, pdc, pds, pdg, ptm, M, E, top_k,
                         1 if renormalize else 0, H, I, po, ot, ids.data_ptr(), weights.data_ptr(),
                         ws.data_ptr() if nw else None, nw, stream)
    if st:
        _lib.check(st, "wush_moe_w4(%s)" % fmt)
    return MoeResult(out, ids, weights)


class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor       # float32 [R]
    entropy: torch.Tensor       # float32 [R], in nats
    top_ids: torch.Tensor       # int32 [R, top]
    top_logprobs: torch.Tensor  # float32 [R, top]


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, top: int = 0) -> TokenLogprobs:
    """Log probabilities of the tokens targets [R] (int64; negative: not
    scored, 0) under logits [R, V] (float32, bfloat16 or float16, rows V or more
    elements apart), the rows' entropies and their `top` most likely tokens (ties to the
    lower id).  Masked tokens (-inf) have probability 0 and are not listed."""
    if logits.dim() != 2:
        raise ValueError("logits must be [R, V]")
    if logits.dtype not in _LOGITS:
        raise TypeError("logits must be float32, bfloat16 or float16 (got %s)" % logits.dtype)
    R, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits must have contiguous rows")
    dev, stream = _enter(logits, "logits")
    lt = _LOGITS[logits.dtype]
    pt = _check(targets, "targets", torch.int64, (R,), dev)
    values = torch.empty((2, R), dtype=torch.float32, device=dev)
    ids = torch.empty((R, max(top, 0)), dtype=torch.int32, device=dev)
    alt = torch.empty((R, max(top, 0)), dtype=torch.float32, device=dev)
    lib = _lib.load()
    nw = lib.wush_token_logprobs_workspace(R, V, lt, top)
    ws = _workspace(nw, dev)
    p = values.data_ptr()
    st = lib.wush_token_logprobs(logits.data_ptr(), lt, logits.stride(0), R, V, pt, top, p, p + 4 * R, ids.data_ptr(),
                                 alt.data_ptr(), ws.data_ptr() if nw else None, nw, stream)
    if st:
        _lib.check(st, "wush_token_logprobs")
    return TokenLogprobs(values[0], values[1], ids, alt)
