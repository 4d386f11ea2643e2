"""Build the HIP shared library libwush.so in-tree for gfx950, and the native
argument marshalling of some of its Python wrappers (host code only).

Usage: python -m mxfp4_activation_amd.build  (or call build()).
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

from . import _lib

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libwush.so")
BINDING = os.path.join(HERE, "_binding.so")
# (those that take longest first)
SOURCES = ["wush_kernels.hip", "wush_w4.hip", "wush_w4_lora.hip", "wush_kv4_int.hip", "wush_kv4_nv.hip", "wush_kv4_mx.hip",
           "wush_moe.hip", "wush_logprobs.hip", "wush_gptq.hip", "wush_build.hip", "wush_gemm.hip", "wush_kv4.hip", "wush_adjust.hip",
           "wush_dequant.hip", "wush_abi.cpp", "wush_decode_abi.cpp", "wush_serving_abi.cpp"]

HIPCC_FLAGS = [
    "-O3",
    "-std=c++17",
    "--offload-arch=gfx950",
    "-fPIC",
    "-shared",
    # Products are rounded before any add: the code and the reference agree
    # on where fp32 rounding happens.
    "-ffp-contract=off",
    # No packed fp32 ops.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # Matrix-core results go to ordinary VGPRs, not accumulation registers,
    # so the quantization code reads them without v_accvgpr_read copies.
    "-mllvm", "-amdgpu-mfma-vgpr-form=true",
    "-Wall",
    "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _binding_needs() -> str:
    """What csrc/binding.cpp cannot be compiled without and is not here, or nothing."""
    try:
        import torch
    except ImportError:
        return "torch"
    if shutil.which(_cxx()[0]) is None:
        return "a C++ compiler (%s)" % _cxx()[0]
    for name, at in (("Python", os.path.join(sysconfig.get_paths()["include"], "Python.h")),
                     ("torch's HIP", os.path.join(os.path.dirname(torch.__file__), "include", "c10", "hip", "HIPStream.h"))):
        if not os.path.exists(at):
            return "%s headers (%s)" % (name, at)
    return ""


def _cxx():
    return os.environ.get("CXX", "g++").split() or ["g++"]


def build_binding(verbose: bool = False) -> Optional[str]:
    """csrc/binding.cpp against this torch's headers.  None where something that it takes is
    not here: the library needs none of it, and the wrappers do without the binding."""
    needs = _binding_needs()
    if needs:
        sys.stderr.write("_binding.so is not built, for want of %s: the wrappers marshal in Python\n" % needs)
        if os.path.exists(BINDING):  # of another build
            os.remove(BINDING)
        return None
    import torch

    at = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp"
    cmd = _cxx() + ["-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
                    '-DBUILT_FOR="%s"' % _lib.built_for(),
                    "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I" + os.path.join(at, "include"),
                    "-I" + os.path.join(at, "include", "torch", "csrc", "api", "include"), "-I/opt/rocm/include",
                    "-I" + sysconfig.get_paths()["include"], "-o", tmp, os.path.join(CSRC, "binding.cpp"),
                    "-L" + os.path.join(at, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    if verbose:
        print(" ".join(cmd), flush=True)
    _run(cmd)
    os.replace(tmp, BINDING)
    return BINDING


def _run(cmd) -> str:
    """Runs a compiler; what it said, or RuntimeError."""
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("%s failed (exit %d)" % (cmd[0], r.returncode))
    return r.stderr


def build(verbose: bool = False, extra_flags=None) -> str:
    """Every source to an object of its own, several at a time, then the library."""
    flags = HIPCC_FLAGS + list(extra_flags or [])
    tmp = LIB + ".tmp"
    jobs = int(os.environ.get("MAX_JOBS", 0)) or min(8, os.cpu_count() or 1)
    with tempfile.TemporaryDirectory() as out, ThreadPoolExecutor(jobs) as pool:
        objects = [os.path.join(out, s + ".o") for s in SOURCES]
        cmds = [[hipcc()] + [f for f in flags if f != "-shared"] + ["-c", os.path.join(CSRC, s), "-o", o]
                for s, o in zip(SOURCES, objects)]
        link = [hipcc()] + flags + ["-o", tmp] + objects
        if verbose:
            for cmd in cmds + [link]:
                print(" ".join(cmd), flush=True)
        said = list(pool.map(_run, cmds)) + [_run(link)]
    if verbose:
        sys.stderr.write("".join(t for t in said if t.strip()))
    os.replace(tmp, LIB)
    build_binding(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
