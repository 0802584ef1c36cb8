"""Build libgb300moe.so in-tree with nvcc for sm_103a (no cmake, no setup.py).

Each ``csrc/*.cu`` file is compiled in parallel to an object file under ``_build/`` and the
objects are linked into ``_build/libgb300moe.so``, which needs nvcc alone; ``csrc/calls.cpp``, the
Python module over some of its calls, goes to ``_build/gb300moe_calls.so`` and needs a host compiler,
Python's headers and torch's.  Each is rebuilt only when a source or header of its own is newer, the
module also for another torch or Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libgb300moe.so")
CALLS = os.path.join(BUILD, "gb300moe_calls.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libgb300moe.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def library_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def _calls_built_for() -> str:
    """What a build of the Python module fits: torch's C++ interface and Python's change between
    versions."""
    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}\n"


def calls_up_to_date() -> bool:
    if not _newer(CALLS, glob.glob(os.path.join(CSRC, "*.cpp")) + _headers()):
        return False
    try:
        with open(CALLS + ".built_for") as f:
            return f.read() == _calls_built_for()
    except OSError:
        return False


def up_to_date() -> bool:
    return library_up_to_date() and calls_up_to_date()


def _compile(nvcc: str, src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_calls(nvcc: str) -> str:
    """The object of the Python module (host code against torch's headers)."""
    import torch
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    tdir = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    obj = os.path.join(BUILD, "calls.o")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-I", tdir,
           "-I", os.path.join(tdir, "torch", "csrc", "api", "include"), "-I", cuda,
           "-I", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "calls.cpp"),
           "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for calls.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    import torch
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = [cxx, "-shared", "-o", tmp, obj, "-L", BUILD, "-l:" + os.path.basename(LIB),
           "-Wl,-rpath,$ORIGIN", "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the Python module failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(tmp, "w") as f:
        f.write(_calls_built_for())
    os.replace(tmp, CALLS + ".built_for")


def _build_library(nvcc: str, verbose: bool) -> None:
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(lambda s: _compile(nvcc, s), srcs))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source and link the shared library; return its path."""
    if force or not library_up_to_date():
        os.makedirs(BUILD, exist_ok=True)
        _build_library(_nvcc(), verbose)
    return LIB


def build_calls(force: bool = False) -> str:
    """Compile the Python module against the library (built first); return its path."""
    build_library()
    if force or not calls_up_to_date():
        _link_calls(_compile_calls(_nvcc()))
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    """Build the library and the Python module, side by side; return the library's path.  The
    library is in place before a module that cannot be built raises."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        stale = force or not calls_up_to_date()
        calls = ex.submit(_compile_calls, _nvcc()) if stale else None
        build_library(force, verbose)
    if calls:
        _link_calls(calls.result())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
