"""Builds the CUDA library in-tree: ``liblinattn.so`` next to this file, for sm_100a only; and the
CPython module that makes the calls of block.py, ``_marshal-<what it was built for>.so``."""
from __future__ import annotations

import hashlib
import importlib.util
import os
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblinattn.so")
SOURCES = [os.path.join(CSRC, "la_api.cu"), os.path.join(CSRC, "block_api.cu")]
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


def _compile(command_to, out: str, verbose: bool) -> str:
    """Runs ``command_to(file)`` with a file beside ``out`` that then takes its place: processes that start
    together, or load ``out`` meanwhile, see a whole file or none."""
    fd, tmp = tempfile.mkstemp(suffix=".so", prefix=".building-", dir=os.path.dirname(out))
    os.close(fd)
    try:
        cmd = command_to(tmp)
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed building {os.path.basename(out)}")
        os.chmod(tmp, 0o755)
        os.replace(tmp, out)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)
    return out


def marshal_path() -> str:
    """The CPython module's file, named after what it has to match: its sources, this Python, this torch."""
    import torch

    h = hashlib.sha256(f"{sysconfig.get_config_var('SOABI')} {torch.__version__}".encode())
    for f in (MARSHAL_SOURCE, os.path.join(ROOT, "include", "la.h")):
        with open(f, "rb") as src:
            h.update(src.read())
    return os.path.join(HERE, f"_marshal-{h.hexdigest()[:16]}.so")


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Builds the CPython module between block.py and the library, unless the one for these sources, this
    Python and this torch is there."""
    out = marshal_path()
    if not force and os.path.exists(out):
        return out
    import torch

    top = os.path.dirname(torch.__file__)
    inc = os.path.join(top, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include") if os.path.isabs(nvcc()) else "/usr/local/cuda/include"
    return _compile(lambda to: [
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I", inc, "-I",
        os.path.join(inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"], "-I",
        os.path.join(ROOT, "include"), "-I", cuda, "-o", to, MARSHAL_SOURCE, "-L", os.path.join(top, "lib"),
        "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], out, verbose)


def load_marshal():
    """The CPython module, built if it is missing."""
    name = __package__ + "._marshal"
    spec = importlib.util.spec_from_file_location(name, build_marshal())
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Builds the CUDA library alone (nvcc; neither torch nor Python headers)."""
    if not force and up_to_date():
        return LIB
    return _compile(command, LIB, verbose)


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)
    build_marshal(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
