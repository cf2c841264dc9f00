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
import sys

import torch

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


def _fresh(made: str, *suffixes: str) -> bool:
    """Is `made` newer than the public header and the sources that end so?"""
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(suffixes)]
    files.append(os.path.join(ROOT, "include", "sigattn.h"))
    return os.path.exists(made) and os.path.getmtime(made) >= max(os.path.getmtime(f) for f in files)


def _binding_stamp() -> str:
    """What the binding is built for besides its source."""
    return f"{sys.version}\ntorch {torch.__version__}\n"


def _binding_fresh() -> bool:
    stamp = os.path.join(BUILD, "binding.stamp")
    if not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read() == _binding_stamp() and _fresh(BINDING, ".cpp")


def build(force: bool = False, verbose: bool = False) -> str:
    """The C library, and after it (compiled beside it) the binding: if that
    fails the library is there all the same."""
    lib, binding = force or not _fresh(LIB, ".cu", ".cuh"), force or not _binding_fresh()
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        obj = ex.submit(_compile_binding) if binding else None
        if lib:
            _link_library(list(ex.map(lambda src: _compile_cuda(src, verbose), SOURCES)))
        if binding:
            _link_binding(obj.result())
    return LIB


def _compile_cuda(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [_nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    out = _run(f"nvcc for {src}", cmd)
    if verbose:
        print(out)
    return obj


def _link_library(objs: list[str]) -> None:
    tmp = LIB + ".tmp"
    _run("link of libsigattn.so", [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)


def _run(what: str, cmd: list[str]) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _compile_binding() -> str:
    """csrc/binding.cpp against this Python's and torch's headers."""
    import sysconfig

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
    with open(os.path.join(BUILD, "binding.stamp"), "w") as f:
        f.write(_binding_stamp())


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
