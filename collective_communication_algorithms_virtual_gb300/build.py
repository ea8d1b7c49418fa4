"""Builds libvcoll.so, the CUDA library behind the C ABI in include/vc.h, and
_lists.so, the part of the Python binding that is compiled.

Compiles for sm_103a only (GB300).  The translation units are compiled in
parallel into ``_build/`` and linked in place next to this file, where the
Python binding loads both.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libvcoll.so")
LISTS, LISTS_SOURCE = os.path.join(PKG, "_lists.so"), os.path.join(CSRC, "lists.cpp")
SOURCES = ["plan.cpp", "vc.cu", "norm.cu", "route.cu", "exchange.cu", "expert.cu", "quantize.cu", "clip.cu"]
HEADERS = ["plan.h", "host.h", "kernels.cuh", "slice.cuh", "layer.cuh", "tc.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    found = shutil.which("nvcc")
    if found:
        return found
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [LISTS_SOURCE, os.path.join(INCLUDE, "vc.h"), __file__]
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(LISTS):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(LISTS))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _lists_command(to: str) -> list:
    """One compiler call: a Python extension against PyTorch's headers."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    include, libs = os.path.join(torch, "include"), os.path.join(torch, "lib")
    return [shutil.which("g++") or "c++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
            "-I", sysconfig.get_paths()["include"], "-I", include, "-I", os.path.join(include, "torch", "csrc", "api", "include"),
            LISTS_SOURCE, "-o", to, "-L", libs, "-lc10", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{libs}"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libvcoll.so and _lists.so if any source is newer;
    returns the library's path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    common = ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I", INCLUDE, "-I", CSRC]
    lists = LISTS + ".tmp"
    procs = [(cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)) for cmd in [_lists_command(lists)]]
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        cmd = [cc, *common, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cu"):
            cmd[1:1] = ["-Xptxas", "-v"] if verbose else []
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    for cmd, p in procs:
        out, _ = p.communicate()
        if verbose and out:
            print(out)
        if p.returncode != 0:
            raise RuntimeError(f"compile failed ({' '.join(cmd)}):\n{out}")
    tmp = LIB + ".tmp"
    link = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed ({' '.join(link)}):\n{r.stdout}")
    os.replace(tmp, LIB)
    os.replace(lists, LISTS)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
