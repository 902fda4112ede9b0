"""What build() makes without PyTorch or its compiler, and when it makes the binding anew."""
import os
import sys
import types

import pytest

from paged_mla_decode_04_gb300 import _build


@pytest.fixture
def small(monkeypatch, tmp_path):
    """A library of one source file, in a folder of its own."""
    monkeypatch.setattr(_build, "SOURCES", ["selftest.cu"])
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    real = _build.binding_path
    monkeypatch.setattr(_build, "binding_path", lambda: str(tmp_path / os.path.basename(real())))
    return lambda: _build.build(lib_path=_build.LIB, build_dir=str(tmp_path / "obj"))


def test_library_without_torch(small, monkeypatch, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert small() == _build.LIB and os.path.exists(_build.LIB)
    assert not [f for f in os.listdir(tmp_path) if "binding" in f]


def test_library_without_the_bindings_compiler(small, monkeypatch):
    for missing in ("false", "/nonexistent/g++"):
        monkeypatch.setenv("CXX", missing)
        with pytest.raises(RuntimeError, match="binding"):
            small()
        assert os.path.exists(_build.LIB)
        os.remove(_build.LIB)


def test_the_binding_belongs_to_a_torch_and_a_python(monkeypatch):
    """One compiled against another version's headers is never taken for this one's."""
    import torch

    import paged_mla_decode_04_gb300 as m
    here = _build.binding_path()
    assert m.BINDING_PATH == here and torch.__version__ in here and sys.implementation.cache_tag in here
    monkeypatch.setattr(torch, "__version__", "9.9.0+cu1")
    other = _build.binding_path()
    assert other != here
    monkeypatch.setattr(sys, "implementation", types.SimpleNamespace(cache_tag="cpython-399"))
    assert _build.binding_path() not in (here, other)


def test_only_what_is_stale_is_made(small, monkeypatch, tmp_path):
    made = []
    monkeypatch.setattr(_build, "_make_binding", lambda target: (made.append(target), open(target, "w").close()))
    small()
    first = os.path.getmtime(_build.LIB)
    small()
    assert made == [str(tmp_path / os.path.basename(_build.binding_path()))] and os.path.getmtime(_build.LIB) == first
