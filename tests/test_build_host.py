"""build(): the library needs nvcc alone.  A PyTorch that cannot be compiled
against costs the Python calls of adaln_ops.h, with a warning, and nothing else."""

from __future__ import annotations

import ctypes
import os
import sys

import pytest

from invariant_dit_adaln_gb300 import binding, build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one short translation unit in a directory of its own."""
    monkeypatch.setattr(build, "SOURCES", ["one.cu"])
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib" / "libadaln.so"))
    monkeypatch.setattr(build, "MARSHAL_SOURCE", str(tmp_path / "csrc" / "marshal.cpp"))
    (tmp_path / "csrc" / "marshal.cpp").write_text('extern "C" int two() { return 2; }\n')
    return tmp_path


def loads():
    return ctypes.CDLL(build.LIB).one() == 1


def test_both(small, recwarn):
    assert build.build() == build.LIB and loads()
    assert ctypes.CDLL(build.marshal_path()).two() == 2 and not recwarn.list
    for part in (sys.implementation.cache_tag, __import__("torch").__version__.split("+")[0].replace(".", "_")):
        assert part in os.path.basename(build.marshal_path())


@pytest.mark.parametrize("how", ["compiler fails", "no compiler", "no PyTorch"])
def test_library_without_the_module(small, monkeypatch, how):
    if how == "no PyTorch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setenv("CXX", "/bin/false" if how == "compiler fails" else str(small / "missing"))
    for _ in range(2):  # also when the library is up to date
        with pytest.warns(RuntimeWarning, match="module behind the Python calls of adaln_ops.h"):
            assert build.build() == build.LIB
        assert loads()


def test_an_outdated_module_is_not_kept(small, monkeypatch):
    """One compiled against other headers must not be called."""
    build.build()
    path = build.marshal_path()
    os.utime(path, (1, 1))
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.warns(RuntimeWarning):
        build.build()
    assert not os.path.exists(path)


def test_calls_without_the_module_raise(small, monkeypatch):
    import torch
    monkeypatch.setattr(binding, "_marshal", None)
    monkeypatch.setattr(binding, "load", lambda: None)
    with pytest.raises(RuntimeError, match="build_marshal"):
        binding.adaln_grad_norm([torch.zeros(3)])
