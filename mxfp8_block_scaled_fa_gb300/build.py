"""Build libmxfa.so in-tree with nvcc for sm_103a (no cmake, parallel TUs), and kv_py.so, the
Python module of the 4-bit cache's calls, with g++.  The library stands without the module."""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libmxfa.so")


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        pass
    try:
        import torch
        return torch.__version__
    except ImportError:
        return "none"


# named by the torch and the interpreter it is built for, whose interfaces it uses
PY_MODULE = os.path.join(OUT, f"kv_py-{_torch_version()}{sysconfig.get_config_var('EXT_SUFFIX') or '.so'}")
PY_SRC = os.path.join(CSRC, "kv_py.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    inc = os.path.join(os.path.dirname(HERE), "include", "mxfa.h")
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hdrs + [inc]


def _fresh(path: str, made_of) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(p) for p in made_of)


def _gxx(args) -> None:
    r = subprocess.run(["g++", *args], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {PY_SRC}:\n{r.stderr}")


def _torch_folder() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    return spec.submodule_search_locations[0]


def _compile_py_module() -> str:
    """kv_py.o, against the installed torch and Python."""
    torch_at = _torch_folder()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(torch_at, "include"), os.path.join(torch_at, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    obj = os.path.join(OUT, "kv_py.o")
    _gxx(["-O2", "-std=c++17", "-fPIC", *[f"-I{i}" for i in inc], "-c", PY_SRC, "-o", obj])
    return obj


def _link_py_module(obj: str) -> None:
    tmp = PY_MODULE + f".tmp{os.getpid()}"
    _gxx(["-shared", "-o", tmp, obj, f"-L{OUT}", "-lmxfa", f"-L{os.path.join(_torch_folder(), 'lib')}", "-ltorch_python",
          "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, PY_MODULE)


def _py_module_fresh() -> bool:
    return _fresh(PY_MODULE, [__file__, PY_SRC, *_deps()])


def _drop_py_module() -> None:
    """An outdated module goes before a new one is tried: it may not fit the library."""
    with contextlib.suppress(FileNotFoundError):
        os.remove(PY_MODULE)


def build_py_module() -> str:
    """The Python module alone, beside a built library; raises where it cannot be built."""
    if not _py_module_fresh():
        _drop_py_module()
        _link_py_module(_compile_py_module())
    return PY_MODULE


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, which raises where it cannot be built, then the Python module, which warns: the
    4-bit cache's Python calls alone need it, and say so when it is missing."""
    os.makedirs(OUT, exist_ok=True)
    srcs = sources()
    new_lib = force or not _fresh(LIB, srcs + _deps() + [__file__])
    new_module = force or not _py_module_fresh()
    py_obj = None
    if new_module:
        _drop_py_module()
    if new_lib:
        nvcc = _nvcc()

        def compile_one(src):
            obj = os.path.join(OUT, os.path.basename(src)[:-3] + ".o")
            cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
            if verbose:
                cmd += ["-Xptxas", "-v"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
            return obj, r.stderr

        with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
            if new_module:  # beside the library's sources
                py_obj = ex.submit(_compile_py_module)
            results = list(ex.map(compile_one, srcs))
        if verbose:
            for _, log in results:
                print(log)
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]], check=True)
        os.replace(tmp, LIB)
    if new_module:
        try:
            _link_py_module(py_obj.result() if py_obj else _compile_py_module())
        except Exception as e:
            warnings.warn(f"{PY_MODULE} was not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
