"""The in-tree build: the CUDA library must not depend on what only the 8-bit cache's Python calls need (g++ beside
nvcc, Python's and torch's headers)."""
import os
import subprocess

import pytest

from fp4_kv_cache_quant_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """One small source and an extension source that compiles, in a folder of their own."""
    cu, py = tmp_path / "one.cu", tmp_path / "py_bdfp8.cpp"
    cu.write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    py.write_text('#include <Python.h>\n#include <torch/csrc/autograd/python_variable.h>\n')
    for name, path in (("LIB", "lib.so"), ("PY_LIB", "ext.so"), ("OBJ", "obj"), ("PY_SRC", "py_bdfp8.cpp")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    monkeypatch.setattr(build, "sources", lambda: [str(cu)])
    monkeypatch.setattr(build, "_headers", lambda: [])
    return tmp_path


def _times(tree):
    return {n: os.path.getmtime(tree / n) for n in ("lib.so", "ext.so") if (tree / n).exists()}


@pytest.mark.parametrize("missing", ["headers", "compiler"])
def test_the_library_is_built_without_the_extension(tree, monkeypatch, missing):
    (tree / "ext.so").write_text("of an older source")
    os.utime(tree / "ext.so", (1, 1))
    if missing == "headers":
        (tree / "py_bdfp8.cpp").write_text("#include <no_such_header.h>\n")
    else:
        run = subprocess.run

        def without(cmd, *a, **kw):
            if cmd[0] == "g++":
                raise FileNotFoundError("g++")
            return run(cmd, *a, **kw)
        monkeypatch.setattr(subprocess, "run", without)
    with pytest.warns(RuntimeWarning, match="8-bit"):
        assert build.build() == str(tree / "lib.so")
    t = _times(tree)
    assert list(t) == ["lib.so"]     # an extension of older sources is not left beside a newer library
    with pytest.warns(RuntimeWarning, match="8-bit"):
        build.build()
    assert _times(tree) == t         # the library is up to date


def test_each_part_is_built_when_it_is_out_of_date(tree):
    build.build()
    t = _times(tree)
    assert len(t) == 2
    build.build()
    assert _times(tree) == t
    os.utime(tree / "py_bdfp8.cpp", (t["ext.so"] + 10,) * 2)
    build.build()
    u = _times(tree)
    assert u["lib.so"] == t["lib.so"] and u["ext.so"] > t["ext.so"]
    os.utime(tree / "one.cu", (u["ext.so"] + 10,) * 2)
    build.build()
    assert _times(tree)["lib.so"] > u["lib.so"]
