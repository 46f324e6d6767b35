"""Builds the CUDA library in-tree: ``liblinattn.so`` next to this file, for sm_100a only; and the
CPython module ``_marshal.so`` that makes the calls of block.py."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblinattn.so")
SOURCES = [os.path.join(CSRC, "la_api.cu"), os.path.join(CSRC, "block_api.cu")]
MARSHAL = os.path.join(HERE, "_marshal.so")
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")] + [
    os.path.join(ROOT, "include", "la.h")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def command(out: str = LIB, extra=()) -> list:
    ptxas = ["-Xptxas", "-v"] if os.environ.get("LA_PTXAS_V") else []
    return [nvcc(), "-std=c++17", "-O3", "-lineinfo",
            "--threads", "0", "-gencode", "arch=compute_100a,code=sm_100a", "-Xcompiler", "-fPIC", "-shared",
            "-cudart", "shared", *ptxas,
            "-I", os.path.join(ROOT, "include"), "-I", CSRC, *extra, "-o", out, *SOURCES]


def build_variant(out: str, defines=(), verbose: bool = False) -> str:
    """Builds the library with extra preprocessor definitions (e.g. the checked build,
    ``LA_CHECKED``, or the test-hooks build) into ``out``."""
    cmd = command(out, extra=[f"-D{d}" for d in defines])
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"nvcc failed building {out}")
    return out


def up_to_date(out: str = LIB) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(f) <= t for f in DEPS)


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Builds the CPython module between block.py and the library, ``_marshal.so``."""
    if not force and os.path.exists(MARSHAL) and all(
            os.path.getmtime(f) <= os.path.getmtime(MARSHAL) for f in (MARSHAL_SOURCE, os.path.join(ROOT, "include", "la.h"))):
        return MARSHAL
    import sysconfig

    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include") if os.path.isabs(nvcc()) else "/usr/local/cuda/include"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I", inc, "-I",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"], "-I",
           os.path.join(ROOT, "include"), "-I", cuda, "-o", MARSHAL, MARSHAL_SOURCE, "-L",
           os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed building _marshal.so")
    return MARSHAL


def build(force: bool = False, verbose: bool = False) -> str:
    build_marshal(force, verbose)
    if not force and up_to_date():
        return LIB
    cmd = command()
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc failed building liblinattn.so")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
