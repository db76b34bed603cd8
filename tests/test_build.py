"""The build's parts: the C library does not need the Python module's toolchain, and the module
is named by what it is built for (CPU only)."""
import ctypes
import importlib.metadata
import importlib.util
import os
import sysconfig
import warnings

import pytest

from mxfp8_block_scaled_fa_gb300 import build as real


@pytest.fixture()
def small(monkeypatch, tmp_path):
    """A build module of its own, with one small source and its own output folder."""
    spec = importlib.util.spec_from_file_location("mxfa_build_copy", real.__file__)
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int answer() { return 42; }\n')
    monkeypatch.setattr(b, "OUT", str(tmp_path / "out"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "out" / "libmxfa.so"))
    monkeypatch.setattr(b, "PY_MODULE", str(tmp_path / "out" / os.path.basename(b.PY_MODULE)))
    monkeypatch.setattr(b, "sources", lambda: [str(src)])
    return b


@pytest.mark.parametrize("at", ["_compile_py_module", "_link_py_module"])
def test_library_without_the_python_module(small, monkeypatch, at):
    def fail(*a):
        raise RuntimeError("no such compiler")
    monkeypatch.setattr(small, "_compile_py_module", lambda *a: "kv_py.o")
    monkeypatch.setattr(small, "_link_py_module", lambda *a: None)
    monkeypatch.setattr(small, at, fail)
    with pytest.warns(RuntimeWarning, match="no such compiler"):
        assert small.build(force=True) == small.LIB
    assert ctypes.CDLL(small.LIB).answer() == 42
    stamp = os.stat(small.LIB).st_mtime_ns
    with pytest.raises(RuntimeError, match="no such compiler"):
        small.build_py_module()                               # asked for by itself it fails
    with pytest.warns(RuntimeWarning):
        small.build()                                         # tried again, without the library
    assert os.stat(small.LIB).st_mtime_ns == stamp


def test_a_failed_library_is_an_error(small, monkeypatch, tmp_path):
    monkeypatch.setattr(small, "_compile_py_module", lambda *a: "kv_py.o")
    (tmp_path / "one.cu").write_text("no source\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        small.build(force=True)


def test_imports_without_package_metadata(monkeypatch):
    def none(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", none)
    spec = importlib.util.spec_from_file_location("mxfa_build_bare", real.__file__)
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    assert b.LIB == real.LIB and b.PY_MODULE.endswith(".so")


def test_module_is_named_by_torch_and_interpreter():
    import torch
    name = os.path.basename(real.PY_MODULE)
    assert torch.__version__.split("+")[0] in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_a_missing_module_is_named(monkeypatch, tmp_path):
    from mxfp8_block_scaled_fa_gb300 import mxfa
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        real.build()
    monkeypatch.setattr(mxfa, "_kv", None)
    monkeypatch.setattr(real, "PY_MODULE", str(tmp_path / "absent.so"))
    mxfa.lib()                                                # the library's calls need none of it
    with pytest.raises(RuntimeError, match="absent.so"):
        mxfa._fast()


@pytest.mark.parametrize("call", ["build", "build_py_module"])
def test_an_outdated_module_does_not_stay(small, monkeypatch, call):
    """A module of older sources may disagree with the new library on its structures."""
    def fail(*a):
        raise RuntimeError("no such compiler")
    monkeypatch.setattr(small, "_compile_py_module", lambda *a: "kv_py.o")
    monkeypatch.setattr(small, "_link_py_module", lambda *a: None)
    small.build()
    with open(small.PY_MODULE, "w") as f:
        f.write("old")
    os.utime(small.PY_MODULE, (1, 1))
    monkeypatch.setattr(small, "_compile_py_module", fail)
    with (pytest.warns(RuntimeWarning) if call == "build" else pytest.raises(RuntimeError)):
        getattr(small, call)()
    assert not os.path.exists(small.PY_MODULE) and os.path.exists(small.LIB)
