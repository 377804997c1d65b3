"""Builds libmoe.so (the C-ABI library) in-tree with nvcc for sm_103a, and _py_call.so
(the binding's call path, csrc/py_call.cpp) with g++ against it.

Each source compiles in parallel to an object under _build/, then the shared
libraries are linked next to this file. A rebuild happens only when a source or
header is newer than its library. libmoe.so needs nvcc alone and is linked first;
_py_call.so also needs g++, Python's headers and torch, reads torch's objects by the layout of
one version, and is made again for another torch or Python. This file run with --library makes
libmoe.so and stops. No CMake; works the same on x86_64 (where it cross-compiles without a GPU)
and on aarch64.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe.so")
PY_CALL = os.path.join(HERE, "_py_call.so")
PY_CALL_SOURCE = os.path.join(CSRC, "py_call.cpp")
PY_CALL_STAMP = "py_call.built_for"  # under BUILD
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or install the CUDA toolkit")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def _newer(lib: str, files) -> bool:
    return os.path.exists(lib) and all(os.path.getmtime(f) <= os.path.getmtime(lib) for f in files)


def library_up_to_date() -> bool:
    return _newer(LIB, [f for f in _inputs() if f != PY_CALL_SOURCE])


def built_for() -> str:
    """What _py_call.so is bound to."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def call_path_up_to_date() -> bool:
    if not _newer(PY_CALL, [f for f in _inputs() if os.path.dirname(f) != CSRC or f == PY_CALL_SOURCE]):
        return False
    try:
        with open(os.path.join(BUILD, PY_CALL_STAMP)) as f:
            return f.read() == built_for()
    except (OSError, ImportError):
        return False


def up_to_date() -> bool:
    return library_up_to_date() and call_path_up_to_date()


def _compile(src: str, extra, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _torch_dir() -> str:
    import torch  # (its headers and libraries, not a device)
    return os.path.dirname(torch.__file__)


def _compile_py_call() -> str:
    import torch
    inc, obj = os.path.join(_torch_dir(), "include"), os.path.join(BUILD, "py_call.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DMOE_BUILT_FOR="{built_for()}"',
           "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-c", PY_CALL_SOURCE, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on py_call.cpp (it needs Python's and torch's headers; "
                           f"libmoe.so does not):\n{r.stdout}\n{r.stderr}")
    return obj


def _link_py_call(obj: str):
    tmp, stamp = PY_CALL + ".tmp", os.path.join(BUILD, PY_CALL_STAMP)
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", HERE, "-l:libmoe.so",
           "-Wl,-rpath,$ORIGIN", "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _py_call.so failed:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(stamp):  # (never beside another module than the one it is of)
        os.remove(stamp)
    os.replace(tmp, PY_CALL)
    with open(stamp, "w") as f:
        f.write(built_for())


def _link_library(objs):
    tmp = LIB + ".tmp"
    r = subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False,
          library_only: bool = False) -> str:
    """Compiles and links libmoe.so and _py_call.so if needed; returns the former's path. Where
    the latter fails, the former stands all the same."""
    library = force or not library_up_to_date()
    call_path = not library_only and (force or not call_path_up_to_date())
    if not (library or call_path):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    srcs = sources() if library else []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        py_call = ex.submit(_compile_py_call) if call_path else None
        if library:
            _link_library(list(ex.map(lambda s: _compile(s, extra, verbose or ptxas_verbose), srcs)))
        if call_path:
            _link_py_call(py_call.result())
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv,
          library_only="--library" in sys.argv)
    print(LIB)
