"""The native marshalling is an addition: the library builds, and the wrappers work, without it (CPU)."""

import sys

import pytest

from mxfp4_activation_amd import build

torch = pytest.importorskip("torch")


@pytest.fixture
def target(monkeypatch, tmp_path):
    """A binding of some other build, in the place of the package's."""
    at = tmp_path / "_binding.so"
    at.write_bytes(b"of another build")
    monkeypatch.setattr(build, "BINDING", str(at))
    return at


@pytest.mark.parametrize("missing", ["torch", "compiler", "Python's headers", "torch's headers"])
def test_what_the_binding_needs_is_not_needed_by_the_library(monkeypatch, capsys, target, tmp_path, missing):
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif missing == "compiler":
        monkeypatch.setenv("CXX", "no-such-compiler -m64")
    elif missing == "Python's headers":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        monkeypatch.setattr(torch, "__file__", str(tmp_path / "__init__.py"))
    assert build.build_binding() is None
    assert not target.exists() and "marshal in Python" in capsys.readouterr().err


def test_a_compiler_that_fails_is_an_error(monkeypatch, target):
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="false failed"):
        build.build_binding()
    assert target.exists()
