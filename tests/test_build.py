"""What the build makes where torch, or another torch, is installed (no GPU; a
stand-in for nvcc, nothing is compiled)."""
import os
import stat

import pytest

import w8_quantized_linear_b200 as bn
from w8_quantized_linear_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree of its own, and compilers that write their -o file."""
    fake = tmp_path / "cc"
    fake.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done\n')
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(fake))
    monkeypatch.setenv("CXX", str(fake))
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libbitnest.so"))
    return tmp_path


def test_library_is_built_without_torch(tree, monkeypatch, capsys):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == str(tree / "libbitnest.so")
    assert os.path.exists(tree / "libbitnest.so") and "torch is not installed" in capsys.readouterr().err
    assert not list(tree.glob("_binding*"))


def test_library_is_built_before_the_binding_fails(tree, monkeypatch):
    monkeypatch.setenv("CXX", str(tree / "missing"))
    with pytest.raises(OSError):
        build.build()
    assert os.path.exists(tree / "libbitnest.so")


def test_binding_is_of_the_torch_that_is_installed(tree, monkeypatch):
    torch = pytest.importorskip("torch")
    old = tree / "_binding.cpython-312-torch1.0.so"
    old.write_text("another's")
    (tree / "_binding.so").write_text("another's")
    path = build.build_binding()
    assert path == build.binding_path(torch.__version__) and os.path.exists(path)
    assert [p.name for p in tree.glob("_binding*")] == [os.path.basename(path)]
    when = os.path.getmtime(path)
    os.utime(path, (when + 5, when + 5))
    assert build.build_binding() == path and os.path.getmtime(path) == when + 5  # kept


def test_binding_of_another_torch_is_not_loaded(monkeypatch):
    torch = pytest.importorskip("torch")
    build.build()
    monkeypatch.setattr(bn, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "1.0")
    with pytest.raises(ImportError, match="torch1.0"):
        bn.kv_read(1, None, 1, None, None)
