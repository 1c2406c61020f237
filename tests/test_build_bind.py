"""The build of the library and of its Python binding, on small stand-ins for the sources:
the library does not depend on the binding's success."""
import os

import pytest

from kimi_delta_attention_rule_gb300 import build as kbuild

GOOD = "#include <Python.h>\nstatic PyModuleDef m = {PyModuleDef_HEAD_INIT, \"x\"};\nPyMODINIT_FUNC PyInit_x() { return PyModule_Create(&m); }\n"


@pytest.fixture
def tree(tmp_path, monkeypatch):
    (tmp_path / "csrc").mkdir()
    (tmp_path / "include").mkdir()
    (tmp_path / "csrc" / "a.cu").write_text("extern \"C\" int answer() { return 42; }\n")
    (tmp_path / "csrc" / "bind.cpp").write_text(GOOD)
    for name, path in (("CSRC", "csrc"), ("INCLUDE", "include"), ("OBJDIR", "_build"), ("LIB", "lib.so"), ("BIND", "x.so"),
                       ("BIND_SRC", "csrc/bind.cpp")):
        monkeypatch.setattr(kbuild, name, str(tmp_path / path))
    return tmp_path


def test_a_binding_that_does_not_compile_leaves_the_library(tree):
    (tree / "csrc" / "bind.cpp").write_text("#error no headers here\n")
    with pytest.warns(UserWarning, match="binding"):
        assert kbuild.build() == kbuild.LIB
    assert os.path.exists(kbuild.LIB) and not os.path.exists(kbuild.BIND)
    with pytest.warns(UserWarning, match="no headers here"):  # an up-to-date library: the binding is tried again
        kbuild.build()
    with pytest.raises(RuntimeError, match="no headers here"):
        kbuild.build_bind()


def test_a_missing_host_compiler_leaves_the_library(tree, monkeypatch):
    monkeypatch.setenv("CXX", str(tree / "no-such-compiler"))
    with pytest.warns(UserWarning, match="binding"):
        kbuild.build()
    assert os.path.exists(kbuild.LIB)


def test_a_library_that_does_not_compile_raises(tree):
    (tree / "csrc" / "a.cu").write_text("#error not this\n")
    with pytest.raises(RuntimeError, match="not this"):
        kbuild.build()


def test_both_are_built_once(tree):
    kbuild.build()
    times = [os.stat(p).st_mtime_ns for p in (kbuild.LIB, kbuild.BIND)]
    kbuild.build()
    assert times == [os.stat(p).st_mtime_ns for p in (kbuild.LIB, kbuild.BIND)]


def test_another_pytorch_or_python_builds_the_binding_anew(tree, monkeypatch):
    import torch
    kbuild.build()
    first = os.stat(kbuild.BIND).st_mtime_ns
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    kbuild.build()
    second = os.stat(kbuild.BIND).st_mtime_ns
    assert second != first
    kbuild.build()
    assert os.stat(kbuild.BIND).st_mtime_ns == second
    monkeypatch.setattr("sys.version", "3.99 (another)")
    kbuild.build()
    assert os.stat(kbuild.BIND).st_mtime_ns != second


def test_a_binding_of_unknown_origin_is_built_anew(tree):
    kbuild.build()
    first = os.stat(kbuild.BIND).st_mtime_ns
    (tree / "_build" / "bind.txt").unlink()
    kbuild.build()
    assert os.stat(kbuild.BIND).st_mtime_ns != first


def test_a_stale_binding_does_not_outlive_a_failed_build(tree):
    kbuild.build()
    (tree / "csrc" / "bind.cpp").write_text("#error changed\n")
    with pytest.warns(UserWarning, match="changed"):
        kbuild.build()
    assert not os.path.exists(kbuild.BIND)
