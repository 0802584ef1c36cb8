"""Build libgb300moe.so in-tree with nvcc for sm_103a (no cmake, no setup.py).

Each ``csrc/*.cu`` file is compiled in parallel to an object file under ``_build/`` and the
objects are linked into ``_build/libgb300moe.so``; ``csrc/calls.cpp``, the Python module over some
of its calls, goes to ``_build/gb300moe_calls.so``.  A rebuild happens only when a source or
header is newer than the two.
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


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(CALLS)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return all(os.path.getmtime(d) <= t for d in _deps())


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


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA source and link the shared library; return its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        calls = ex.submit(_compile_calls, nvcc)
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
    _link_calls(calls.result())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
