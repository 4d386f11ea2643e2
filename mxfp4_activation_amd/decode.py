"""Decoding with 4-bit weights: linear layers, with low-rank adapters or without,
and mixtures of experts for a few tokens; penalties, biases and masks on logits,
and the log probabilities of tokens.

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


class LoraAdapters(NamedTuple):
    """Low-rank adapters of one layer: A bf16 [adapters, rank, K], B bf16 [adapters, N,
    rank] (rank a multiple of 8; pad with zeros) and their scales, float32 [adapters]."""
    A: torch.Tensor
    B: torch.Tensor
    scale: Optional[torch.Tensor] = None


def linear_w4_lora(fmt: str, x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, adapters: LoraAdapters,
                   ids: torch.Tensor, T: Optional[torch.Tensor] = None, global_scale: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``linear_w4`` plus each token's own low-rank adapter: x' W^T + scale[e] (x A[e]^T)
    B[e]^T with e = ids[m] (int32 [M]; negative: no adapter, out of range: NaN) and x
    untransformed.  The sums are fp32 and rounded once."""
    native = _lib.binding()
    if native is not None and out_dtype in _OUT:
        r = native.lora(fmt, x, codes, scales, *adapters, ids, T, global_scale, out_dtype is torch.float32, out)
        if r is not None:
            if type(r) is int:
                _lib.check(r, "wush_linear_w4_lora(%s)" % fmt)
            return r
    f, G = _fmt(fmt)
    ot = _out_type(out_dtype)
    M, K, ldx = _rows(x, "x")
    dev, stream = _enter(x, "x")
    if codes.dim() != 2 or adapters.A.dim() != 3:
        raise ValueError("codes must be 2-D and adapters.A [adapters, rank, K]")
    N, (E, rank) = codes.shape[0], adapters.A.shape[:2]
    pc = _check(codes, "codes", torch.uint8, (N, K // 2), dev)
    ps = _check(scales, "scales", _scale_dtype(fmt), (N, K // G), dev)
    pg, global_scale = _check_global(fmt, global_scale, "global_scale", 1, dev)
    pt = None if T is None else _check(T, "T", torch.bfloat16, (K // G, G, G), dev)
    pa = _check(adapters.A, "adapters.A", torch.bfloat16, (E, rank, K), dev)
    pb = _check(adapters.B, "adapters.B", torch.bfloat16, (E, N, rank), dev)
    pe = None if adapters.scale is None else _check(adapters.scale, "adapters.scale", torch.float32, (E,), dev)
    pi = _check(ids, "ids", torch.int32, (M,), dev)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
        po = out.data_ptr()
    else:
        po = _check(out, "out", out_dtype, (M, N), dev)
    lib = _lib.load()
    nw = lib.wush_linear_w4_lora_workspace(M, N, K, rank, 0 if T is None else 1, ot)
    ws = _workspace(nw, dev)
    st = lib.wush_linear_w4_lora(f, x.data_ptr(), ldx, pt, pc, ps, pg, pa, pb, pe, pi, E, rank, M, N, K, po, ot,
                                 ws.data_ptr() if nw else None, nw, stream)
    if st:
        _lib.check(st, "wush_linear_w4_lora(%s)" % fmt)
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


def _logits(logits: torch.Tensor, name: str):
    """(rows, vocabulary, type) of logits whose rows are contiguous."""
    if logits.dim() != 2:
        raise ValueError("%s must be [R, V]" % name)
    if logits.dtype not in _LOGITS:
        raise TypeError("%s must be float32, bfloat16 or float16 (got %s)" % (name, logits.dtype))
    R, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    return R, V, _LOGITS[logits.dtype]


def adjust_logits(logits: torch.Tensor, prompt: Optional[torch.Tensor] = None, output: Optional[torch.Tensor] = None,
                  repetition: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                  presence: Optional[torch.Tensor] = None, bias_ids: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, allowed: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Penalties, biases and grammar masks on logits [R, V] (float32, bfloat16 or
    float16, rows V or more elements apart), in this order: tokens in prompt or output
    (int32 [R, any], -1 pads) are divided (l > 0) or multiplied by repetition [R]; tokens
    in output lose frequency [R] per occurrence and presence [R] once; bias [R, n] is added at
    bias_ids [R, n] (int32, -1 pads); tokens whose bit of allowed (int32 [R, (V + 31) // 32],
    bit v % 32 of word v // 32) is not set become -inf.  The penalties and biases are float32.
    Returns a new tensor, or out, which may be logits itself."""
    native = _lib.binding()
    if native is not None:
        r = native.adjust(logits, prompt, output, repetition, frequency, presence, bias_ids, bias, allowed, out)
        if r is not None:
            if type(r) is int:
                _lib.check(r, "wush_adjust_logits")
            return r
    R, V, lt = _logits(logits, "logits")
    dev, stream = _enter(logits, "logits")

    def table(t, name, dtype):
        if t is None:
            return None, 0
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError("%s must be a tensor [R, n]" % name)
        return _check(t, name, dtype, (R, t.shape[1]), dev), t.shape[1]

    def row(t, name):
        return None if t is None else _check(t, name, torch.float32, (R,), dev)

    pp, n_prompt = table(prompt, "prompt", torch.int32)
    po, n_output = table(output, "output", torch.int32)
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    pi, n_bias = table(bias_ids, "bias_ids", torch.int32)
    pb = None if bias is None else _check(bias, "bias", torch.float32, (R, n_bias), dev)
    pm = None if allowed is None else _check(allowed, "allowed", torch.int32, (R, (V + 31) // 32), dev)
    if out is None:
        out = torch.empty((R, V), dtype=logits.dtype, device=dev)
    elif out is not logits:
        if out.shape != logits.shape or out.dtype != logits.dtype or out.device != dev:
            raise ValueError("out must have the shape, type and device of logits")
        _logits(out, "out")
    st = _lib.load().wush_adjust_logits(logits.data_ptr(), lt, logits.stride(0), R, V, pp, n_prompt, po, n_output,
                                        row(repetition, "repetition"), row(frequency, "frequency"),
                                        row(presence, "presence"), pi, pb, n_bias, pm, out.data_ptr(), out.stride(0),
                                        stream)
    if st:
        _lib.check(st, "wush_adjust_logits")
    return out


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
    R, V, lt = _logits(logits, "logits")
    dev, stream = _enter(logits, "logits")
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
