"""Build libmxfa.so in-tree with nvcc for sm_103a (no cmake, parallel TUs), and kv_py.so, the
Python module of the 4-bit cache's calls, with g++."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libmxfa.so")
# named by the torch it is built for, whose C++ interface it uses
PY_MODULE = os.path.join(OUT, f"kv_py-{importlib.metadata.version('torch')}.so")
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


def _compile_py_module(nvcc: str) -> str:
    """kv_py.o, against the installed torch and Python."""
    torch_at = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    inc = [os.path.join(torch_at, "include"), os.path.join(torch_at, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    obj = os.path.join(OUT, "kv_py.o")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", *[f"-I{i}" for i in inc], "-c", PY_SRC, "-o", obj],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {PY_SRC}:\n{r.stderr}")
    return obj


def _link_py_module(obj: str) -> None:
    libs = os.path.join(importlib.util.find_spec("torch").submodule_search_locations[0], "lib")
    tmp = PY_MODULE + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{OUT}", "-lmxfa", f"-L{libs}", "-ltorch_python", "-ltorch_cuda",
                    "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, PY_MODULE)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT, exist_ok=True)
    srcs = sources()
    newest = max(os.path.getmtime(p) for p in srcs + _deps() + [__file__, PY_SRC])
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= newest for p in (LIB, PY_MODULE)):
        return LIB
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

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        py_obj = ex.submit(_compile_py_module, nvcc)
        results = list(ex.map(compile_one, srcs))
        py_obj = py_obj.result()
    if verbose:
        for _, log in results:
            print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]], check=True)
    os.replace(tmp, LIB)
    _link_py_module(py_obj)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
