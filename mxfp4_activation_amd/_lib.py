"""ctypes loader for libwush.so (the C ABI declared in include/wush.h).

The library is loaded from this package directory.  There is no fallback:
if it has not been built, importing the ops raises.
"""

from __future__ import annotations

import ctypes
import os
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libwush.so")
BINDING_PATH = os.path.join(HERE, "_binding.so")

WUSH_OK, WUSH_EINVAL, WUSH_EALIGN, WUSH_EUNSUPPORTED, WUSH_EHIP = range(5)
FMT = {"mxfp4": 0, "nvfp4": 1, "int4": 2}

# name -> (restype, argtypes); every entry point declared in include/wush.h
_c_int, _i64, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
SIGNATURES = {
    "wush_quant_mxfp4": (_c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp]),
    "wush_quant_nvfp4": (_c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "wush_quant_int4": (_c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp]),
    "wush_quant": (_c_int, [_c_int, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "wush_gemm_mxfp4": (_c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _c_int, _vp]),
    "wush_gemm_mxfp4_packed": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _i64, _i64, _i64, _vp, _c_int, _vp]),
    "wush_quant_mxfp4_packed": (_c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp]),
    "wush_gemm_pack_b": (_c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp]),
    "wush_dequant": (_c_int, [_c_int, _vp, _vp, _vp, _i64, _i64, _vp, _vp]),
    "wush_gptq_block": (_c_int, [_c_int, _vp, _vp, _c_int, _i64, _vp, _vp, _i64, _vp, _i64, _vp]),
    "wush_gptq_wush": (_c_int, [_c_int, _vp, _vp, _i64, _i64, _i64, _c_int, ctypes.c_double, _c_int, _vp, _vp, _vp,
                                _vp, _vp, _vp, _vp]),
    "wush_build_transforms": (_c_int, [_vp, _i64, _vp, _i64, _i64, _c_int, ctypes.c_double, _c_int, _vp, _vp, _vp,
                                       _vp, _vp]),
    "wush_transform_f32": (_c_int, [_vp, _vp, _i64, _i64, _c_int, _vp, _vp]),
    "wush_absmax_transformed": (_c_int, [_vp, _vp, _i64, _i64, _c_int, _vp, _vp]),
    "wush_fixed_transforms": (_c_int, [_c_int, _i64, _c_int, _vp, _vp, _vp]),
    "wush_f64_to_bf16": (_c_int, [_vp, _i64, _vp, _vp]),
    "wush_nvfp4_global_scale": (_c_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "wush_e2m1_encode": (_c_int, [_vp, _i64, _vp, _vp]),
    "wush_linear_w4": (_c_int, [_c_int, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _c_int, _vp, _i64, _vp]),
    "wush_linear_w4_workspace": (_i64, [_i64, _i64, _c_int]),
    "wush_moe_w4": (_c_int, [_c_int, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _c_int, _c_int,
                             _i64, _i64, _vp, _c_int, _vp, _vp, _vp, _i64, _vp]),
    "wush_moe_w4_workspace": (_i64, [_i64, _i64, _c_int, _i64, _i64, _c_int, _c_int]),
    "wush_token_logprobs": (_c_int, [_vp, _c_int, _i64, _i64, _i64, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _i64, _vp]),
    "wush_token_logprobs_workspace": (_i64, [_i64, _i64, _c_int, _c_int]),
    "wush_kv4_append": (_c_int, [_c_int, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp,
                                 _vp, _vp, _vp, _vp, _vp]),
    "wush_kv4_attention": (_c_int, [_c_int, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp,
                                    _i64, _i64, _i64, _i64, _i64, _i64, _i64, ctypes.c_float, _i64, _vp, _vp, _i64,
                                    _vp]),
    "wush_kv4_attention_workspace": (_i64, [_c_int, _i64, _i64, _i64, _i64, _i64, _i64, _i64]),
    "wush_linear_w4_lora": (_c_int, [_c_int, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                     _i64, _vp, _c_int, _vp, _i64, _vp]),
    "wush_linear_w4_lora_workspace": (_i64, [_i64, _i64, _i64, _i64, _c_int, _c_int]),
    "wush_adjust_logits": (_c_int, [_vp, _c_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64,
                                    _vp, _vp, _i64, _vp]),
    "wush_status_string": (ctypes.c_char_p, [_c_int]),
    "wush_last_error": (ctypes.c_char_p, []),
    "wush_abi_version": (_c_int, []),
}

ABI_VERSION = 2


class WushError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__("%s failed: status %d (%s)" % (where, status, detail))
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Load libwush.so once; raise if it is missing or has the wrong ABI."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libwush.so is not built (%s); run `python -m mxfp4_activation_amd.build`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.wush_abi_version() != ABI_VERSION:
        raise ImportError("libwush.so ABI version mismatch")
    _lib = lib
    return lib


_NATIVE = ("wush_kv4_append", "wush_kv4_attention", "wush_kv4_attention_workspace", "wush_linear_w4_lora",
           "wush_linear_w4_lora_workspace", "wush_adjust_logits", "wush_dequant")
_binding = False  # not looked for yet


def built_for() -> str:
    """What a binding has to have been built for."""
    import torch

    return "torch %s, Python %d.%d, ABI %d" % (torch.__version__, *sys.version_info[:2], ABI_VERSION)


def binding():
    """The native form of the wrappers' argument marshalling (csrc/binding.cpp), or None
    where it is not built: the wrappers then do it in Python, some ten microseconds slower.
    One that cannot be loaded, or was built for something else, is left aside with a
    warning.  Needs torch to be imported."""
    global _binding
    if _binding is False:
        module, why = None, ""
        try:
            from . import _binding as module
        except ImportError as e:
            why = "cannot be loaded (%s)" % e if os.path.exists(BINDING_PATH) else ""
        if module is not None:
            made_for = getattr(module, "built_for", "something else")
            if made_for != built_for():
                module, why = None, "was built for %s, this is %s" % (made_for, built_for())
        if why:
            warnings.warn("_binding.so %s: the wrappers marshal in Python; run `python -m mxfp4_activation_amd.build`" % why,
                          RuntimeWarning, stacklevel=3)
        if module is not None:
            lib = load()
            module.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _NATIVE})
        _binding = module
    return _binding


def check(status: int, where: str) -> None:
    if status != WUSH_OK:
        lib = load()
        detail = lib.wush_last_error().decode() or lib.wush_status_string(status).decode()
        raise WushError(status, where, detail)
