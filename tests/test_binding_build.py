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


@pytest.fixture
def loading(monkeypatch):
    """_lib as it is before the first look for the binding, and f(module or None): what is there to import."""
    import mxfp4_activation_amd as wush
    from mxfp4_activation_amd import _lib

    monkeypatch.setattr(_lib, "_binding", False)
    monkeypatch.delattr(wush, "_binding", raising=False)
    return _lib, lambda module: monkeypatch.setitem(sys.modules, "mxfp4_activation_amd._binding", module)


class _Module:
    def __init__(self, **kw):
        self.bound = None
        self.__dict__.update(kw)

    def bind(self, entries):
        self.bound = entries


def test_a_binding_of_this_build_is_taken(loading, recwarn):
    lib, there = loading
    module = _Module(built_for=lib.built_for())
    there(module)
    assert lib.binding() is module and set(module.bound) == set(lib._NATIVE) and all(module.bound.values())
    assert lib.binding() is module and not recwarn.list


@pytest.mark.parametrize("made", [{}, {"built_for": "torch 0.1, Python 2.7, ABI 1"}])
def test_a_binding_of_another_build_is_left_aside(loading, made):
    lib, there = loading
    module = _Module(**made)
    there(module)
    with pytest.warns(RuntimeWarning, match="was built for"):
        assert lib.binding() is None
    assert module.bound is None


def test_a_binding_that_does_not_load_says_so(loading, monkeypatch, tmp_path):
    lib, there = loading
    there(None)  # an ImportError
    monkeypatch.setattr(lib, "BINDING_PATH", str(tmp_path / "_binding.so"))
    import warnings

    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert lib.binding() is None  # not built: nothing to say
    lib._binding = False
    (tmp_path / "_binding.so").write_bytes(b"?")
    with pytest.warns(RuntimeWarning, match="cannot be loaded"):
        assert lib.binding() is None


def test_the_built_binding_is_of_this_build():
    import os

    from mxfp4_activation_amd import _lib

    if not os.path.exists(_lib.BINDING_PATH):
        pytest.skip("not built")
    from mxfp4_activation_amd import _binding

    assert _binding.built_for == _lib.built_for()
