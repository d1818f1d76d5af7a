"""What build() makes with and without what the Python module needs, on sources of a few lines."""
import ctypes
import os

import pytest

from bidirectional_lstm_stack_gb300 import build as build_mod


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build()'s folders, with a library and a module of one function each."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "some.h").write_text("int lstm_seven(void);\n")
    (csrc / "library.cu").write_text('extern "C" int lstm_seven() { return 7; }\n')
    (csrc / "module.cpp").write_text('extern "C" int lstm_seven();\n'
                                     'extern "C" int module_seven() { return lstm_seven(); }\n')
    for name, value in (("CSRC", csrc), ("PKG", tmp_path), ("BUILD", tmp_path / "_build"),
                        ("LIB", tmp_path / "liblstmstack.so"), ("NATIVE", tmp_path / "_native.so")):
        monkeypatch.setattr(build_mod, name, str(value))
    return tmp_path


def _library_works(tree):
    return ctypes.CDLL(str(tree / "liblstmstack.so")).lstm_seven() == 7


@pytest.fixture
def torch_is_not_installed(monkeypatch):
    find = build_mod.importlib.util.find_spec
    monkeypatch.setattr(build_mod.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))


def test_without_torch_the_library_is_built(tree, torch_is_not_installed):
    with pytest.warns(RuntimeWarning, match="_native.so.* is not: torch is not installed"):
        assert build_mod.build() == str(tree / "liblstmstack.so")
    assert _library_works(tree) and not (tree / "_native.so").exists()


def test_without_python_headers_the_library_is_built(tree, monkeypatch):
    monkeypatch.setattr(build_mod.sysconfig, "get_paths", lambda: {"include": str(tree)})
    with pytest.warns(RuntimeWarning, match="_native.so.* is not: there is no Python.h"):
        build_mod.build()
    assert _library_works(tree) and not (tree / "_native.so").exists()


def test_without_cuda_in_torch_the_library_is_built(tree, monkeypatch):
    (tree / "torch").mkdir()
    monkeypatch.setattr(build_mod, "_torch", lambda: str(tree / "torch"))
    with pytest.warns(RuntimeWarning, match="_native.so.* is not: the torch in .* without CUDA"):
        build_mod.build()
    assert _library_works(tree) and not (tree / "_native.so").exists()


def test_a_module_that_does_not_compile_comes_after_the_library(tree):
    (tree / "csrc" / "module.cpp").write_text("#error no module\n")
    with pytest.raises(RuntimeError, match="no module"):
        build_mod.build()
    assert _library_works(tree) and not (tree / "_native.so").exists()


def test_a_library_that_does_not_compile_is_an_error(tree):
    (tree / "csrc" / "library.cu").write_text("#error no library\n")
    with pytest.raises(RuntimeError, match="no library"):
        build_mod.build()
    assert not (tree / "liblstmstack.so").exists()


def test_only_what_is_old_is_built_again(tree):
    build_mod.build()
    lib, native = (tree / "liblstmstack.so").stat(), (tree / "_native.so").stat()
    build_mod.build()
    assert (tree / "liblstmstack.so").stat().st_mtime_ns == lib.st_mtime_ns
    later = os.path.getmtime(tree / "_build" / "module.o") + 10
    os.utime(tree / "csrc" / "module.cpp", (later, later))
    build_mod.build()
    assert (tree / "liblstmstack.so").stat().st_mtime_ns == lib.st_mtime_ns
    assert (tree / "_native.so").stat().st_mtime_ns > native.st_mtime_ns
