"""What the compiler made of the copies from global memory to LDS, read from the
built library's own gfx950 code (CPU).

The 4-bit products (linear_kernel, gate_up_kernel, down_kernel) copy activations
into LDS behind the compiler's back and publish them by a barrier: a wave may
read what another wave's copy wrote once that wave has waited for it and both have
met.  A copy is issued before one barrier and read after the next, so on every
path its own wave has to have waited for it (s_waitcnt vmcnt) before it reaches
the second barrier behind it; only then does the barrier tell the others
anything.  Memory operations complete in the order of their issue, and vmcnt(n)
leaves at most the n newest of them: a copy with k newer ones has landed if n <= k.

Where paths meet, a copy counts as on its way if it is so on any of them, but k as the
most of them: the loads of weights behind a copy are skipped on the same
conditions (the loop's end, one chunk only) as what follows them, which the paths of
a flow graph do not know.

A copy takes its place in LDS from M0.  Between a scalar write of M0 and a load to
LDS this family's instruction set wants one wait state, which the compiler puts there
for its own pairs but not inside a statement of assembly.
"""

import re

import pytest

from tests import device_code

pytestmark = pytest.mark.skipif(device_code.objdump() is None, reason="llvm-objdump not available")

_VMEM = re.compile(r"^(global|flat|buffer|scratch)_")
_VMCNT = re.compile(r"vmcnt\((\d+)\)")
_MOST = 64  # vmcnt counts no further


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    found = device_code.functions(tmp_path_factory.mktemp("code"))
    assert found, "no gfx950 code in the library"
    return found


def _step(state, i):
    """(state behind instruction i, whether an awaited copy is missing at it).  The state
    (a, b): memory operations issued after the newest copy that may still be on its
    way and has no (a) or one (b) barrier behind it; None: no such copy."""
    a, b = state
    if i.op == "s_waitcnt":
        m = _VMCNT.search(i.args)
        if m:
            n = int(m.group(1))
            a, b = (None if k is None or n <= k else k for k in (a, b))
    elif i.op == "s_barrier":
        return (None, a), b is not None
    elif _VMEM.match(i.op):
        a, b = (None if k is None else min(k + 1, _MOST) for k in (a, b))
        if "load_lds" in i.op:
            a = 0
    return (a, b), False


def _join(s, t):
    if s is None:
        return t
    return tuple(x if y is None else y if x is None else max(x, y) for x, y in zip(s, t))


def unawaited(code):
    """Addresses of barriers that a copy may reach as its second without having been waited for."""
    index = {i.address: n for n, i in enumerate(code)}
    before, todo = {0: (None, None)}, [0]
    while todo:
        n = todo.pop()
        state, _ = _step(before[n], code[n])
        after = [] if code[n].op in ("s_endpgm", "s_branch") else [n + 1]
        if code[n].target is not None:
            after.append(index[code[n].target])
        for m in after:
            joined = _join(before.get(m), state)
            if m < len(code) and joined != before.get(m):
                before[m] = joined
                todo.append(m)
    # The counts grew while the paths were followed: judge by the final ones.
    return {code[n].address for n, state in before.items() if _step(state, code[n])[1]}


def test_the_check_itself():
    def code(*lines):
        return [device_code.Instruction(4 * n, *(line.split(" ", 1) + [""])[:2], t) for n, (line, t) in enumerate(lines)]

    copy, load, barrier, end = ("global_load_lds_dwordx4 v[0:1], off", None), ("global_load_dwordx4 v", None), (
        "s_barrier", None), ("s_endpgm", None)
    wait = [("s_waitcnt vmcnt(%d)" % n, None) for n in range(3)]
    assert not unawaited(code(copy, barrier, wait[0], barrier, end))
    assert unawaited(code(copy, barrier, barrier, end)) == {8}
    assert not unawaited(code(copy, barrier, load, wait[1], barrier, end))
    assert unawaited(code(copy, barrier, load, wait[2], barrier, end)) == {16}
    # One of two paths has no wait.
    assert unawaited(code(copy, barrier, ("s_cbranch_scc0 1", 16), wait[0], barrier, end)) == {16}
    # A loop whose copies are waited for one turn later, and one where they are not.
    assert not unawaited(code(wait[1], copy, barrier, load, ("s_cbranch_scc0 0", 0), end))
    assert unawaited(code(wait[2], copy, barrier, load, ("s_cbranch_scc0 0", 0), end)) == {8}


@pytest.mark.parametrize("kernel", ["linear_kernel", "gate_up_kernel", "down_kernel"])
def test_copies_are_waited_for_before_they_are_published(functions, kernel):
    mine = {name: code for name, code in functions.items() if kernel in name}
    assert mine and all(any("load_lds" in i.op for i in code) for code in mine.values())
    missing = {name: sorted(unawaited(code)) for name, code in mine.items()}
    missing = {name: at for name, at in missing.items() if at}
    assert not missing, "%d of %d kernels: %s" % (len(missing), len(mine), missing)


def test_no_copy_directly_behind_a_write_of_its_base(functions):
    copies, bare = 0, {}
    for name, code in functions.items():
        for before, i in zip(code, code[1:]):
            if "load_lds" in i.op:
                copies += 1
                if before.op.startswith("s_") and re.match(r"m0\b", before.args):
                    bare[name] = bare.get(name, 0) + 1
    assert copies and not bare, bare
