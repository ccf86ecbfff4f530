"""The build's own logic, on a copy of one small source (no GPU needed)."""
import importlib
import os
import shutil

import pytest
import torch

b = importlib.import_module("combine_get_dispatch_layout_gb300.build")   # (the package's `build` is the function)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build() that works under tmp_path: one source, and a binding that counts how often it is built."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    built = []

    def bind():
        built.append(1)
        (tmp_path / "bind.so").write_text("")
        (tmp_path / "stamp").write_text(b._bind_against())

    for name, path in (("LIB", "lib.so"), ("BIND", "bind.so"), ("OBJ", "obj"), ("BIND_STAMP", "stamp")):
        monkeypatch.setattr(b, name, str(tmp_path / path), raising=False)
    monkeypatch.setattr(b, "sources", lambda: [str(src)])
    monkeypatch.setattr(b, "_build_bind", bind)
    return tmp_path, built


def test_the_library_is_built_where_the_binding_cannot_be(tree, monkeypatch):
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("needs nvcc")
    path, _ = tree

    def no_headers():
        raise RuntimeError("Python.h: No such file or directory")

    monkeypatch.setattr(b, "_build_bind", no_headers)
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert b.build() == str(path / "lib.so")
    assert os.path.getsize(path / "lib.so") > 0


def test_another_torch_makes_the_binding_stale(tree, monkeypatch):
    path, built = tree
    (path / "lib.so").write_text("")
    os.utime(path / "one.cu", (0, 0))
    monkeypatch.setattr(b, "INCLUDE", str(path))
    monkeypatch.setattr(b, "CSRC", str(path))
    b.build()
    b.build()
    assert len(built) == 1
    monkeypatch.setattr(torch, "__version__", "99.0")
    b.build()
    b.build()
    assert len(built) == 2
