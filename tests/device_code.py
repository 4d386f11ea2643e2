"""The device code of the built library as instructions, for checks of what the
compiler made of the kernels (CPU; no GPU needed)."""

from __future__ import annotations

import os
import re
import shutil
import struct
import subprocess
from typing import Dict, List, NamedTuple, Optional

from mxfp4_activation_amd import _lib, build

_MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


class Instruction(NamedTuple):
    address: int
    op: str
    args: str
    target: Optional[int]  # of a branch


def objdump() -> Optional[str]:
    """llvm-objdump of the compiler that builds the library, if there is one."""
    try:
        at = os.path.dirname(os.path.realpath(build.hipcc()))
    except RuntimeError:
        return None
    for d in (os.path.join(at, "..", "llvm", "bin"), os.path.join(at, "..", "lib", "llvm", "bin"), at):
        tool = os.path.join(d, "llvm-objdump")
        if os.path.exists(tool):
            return tool
    return shutil.which("llvm-objdump")


def code_objects(lib: str = _lib.LIB_PATH) -> List[bytes]:
    """The gfx950 code objects of the offload bundles in the library."""
    with open(lib, "rb") as f:
        data = f.read()
    found, at = [], data.find(_MAGIC)
    while at >= 0:
        (n,) = struct.unpack_from("<Q", data, at + len(_MAGIC))
        entry = at + len(_MAGIC) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            if b"gfx950" in data[entry + 24 : entry + 24 + length]:
                found.append(data[at + offset : at + offset + size])
            entry += 24 + length
        at = data.find(_MAGIC, entry)
    return found


_HEAD = re.compile(r"^[0-9a-f]+ <(.+)>:$")
_LINE = re.compile(r"^\s+(\S+)(.*?)\s*// ([0-9A-F]+):")


def functions(tmp_path) -> Dict[str, List[Instruction]]:
    """Instructions of every device function by its (mangled) name."""
    tool, out = objdump(), {}
    for i, code in enumerate(code_objects()):
        path = os.path.join(str(tmp_path), "%d.co" % i)
        with open(path, "wb") as f:
            f.write(code)
        text = subprocess.run([tool, "-d", path], capture_output=True, text=True, check=True).stdout
        body = []
        for line in text.splitlines():
            head = _HEAD.match(line)
            if head:
                body = out.setdefault(head.group(1), [])
                continue
            m = _LINE.match(line)
            if not m:
                continue
            op, args, address = m.group(1), m.group(2).strip(), int(m.group(3), 16)
            target = None
            if op.startswith(("s_cbranch", "s_branch")):
                words = int(args)
                target = address + 4 + 4 * (words - 65536 if words >= 32768 else words)
            body.append(Instruction(address, op, args, target))
    return out


def metadata() -> Dict[str, Dict[str, int]]:
    """What the compiler notes of every kernel (registers, spills, scratch) by its (mangled) name."""
    tool, out = os.path.join(os.path.dirname(objdump()), "llvm-readelf"), {}
    for code in code_objects():
        text = subprocess.run([tool, "--notes", "-"], input=code, capture_output=True, check=True).stdout.decode()
        for part in text.split("  - .agpr_count:")[1:]:
            name = re.search(r"^    \.name:\s+(\S+)", part, re.M).group(1)
            out[name] = {k: int(v) for k, v in re.findall(r"^    \.(\w+):\s+(\d+)$", part, re.M)}
    return out
