"""Build the CUDA library ``libsigattn.so`` in-tree with nvcc for sm_100a, and the
Python binding of the paged calls ``_binding.so`` with g++.

Usage: ``python -m sigmoid_attention_b200.build`` (or ``build()`` from Python).
Objects go to ``_build/`` next to the package; the shared library is written
into the package directory so that it ships with the source tree.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsigattn.so")
BINDING = os.path.join(PKG, "_binding.so")
SOURCES = ["api.cu", "plan.cu", "fwd.cu", "bwd.cu", "noalloc.cu", "pages.cu", "paged_few.cu", "paged_many.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".cpp"))]
    return files + [os.path.join(ROOT, "include", "sigattn.h")]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB) and os.path.exists(BINDING):
        newest = max(os.path.getmtime(f) for f in _deps())
        if min(os.path.getmtime(LIB), os.path.getmtime(BINDING)) >= newest:
            return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding_obj = binding.result()
    tmp = LIB + ".tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding_obj)
    return LIB


def _run(what: str, cmd: list[str]) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_binding() -> str:
    """csrc/binding.cpp against this Python's and torch's headers."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    obj = os.path.join(BUILD, "binding.o")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    includes = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    _run("g++ for binding.cpp", [
        "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        *[x for i in includes for x in ("-isystem", i)], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj])
    return obj


def _link_binding(obj: str) -> None:
    from torch.utils import cpp_extension

    tmp = BINDING + ".tmp"
    _run("link of _binding.so", [
        "g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libsigattn.so", "-Wl,-rpath,$ORIGIN",
        *[x for d in cpp_extension.library_paths() for x in ("-L", d)], "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
