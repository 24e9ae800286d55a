"""Builds libsigattn.so in-tree with nvcc for sm_100a (no GPU needed to build),
and ``_calls.so``, the Python entry points of the calls made once per token or
layer, with the host compiler against this PyTorch.

Every ``csrc/*.cu`` file is one translation unit; they compile side by side
into ``_build/`` and are linked into one library.  A unit is compiled again
when it or any header is newer than its object file."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
OUT = os.path.join(HERE, "libsigattn.so")
CALLS_SRC = os.path.join(CSRC, "binding.cpp")
CALLS_OUT = os.path.join(HERE, "_calls.so")
UNITS = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))
HEADERS = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")] + [
    os.path.join(ROOT, "include", "sigattn.h")]
DEPS = [os.path.join(CSRC, f) for f in UNITS] + HEADERS


def _nvcc() -> list[str]:
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-Xcompiler", "-fPIC"]


def compile_cmd(unit: str, obj: str, extra=()) -> list[str]:
    return _nvcc() + ["-lineinfo", "-O3", "-std=c++20", "--expt-relaxed-constexpr",
                      "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, unit), "-o", obj, *extra]


def link_cmd(objs, out: str = OUT) -> list[str]:
    return _nvcc() + ["-shared", *objs, "-o", out]


def calls_cmd(out: str = CALLS_OUT) -> list[str]:
    """Compiles binding.cpp against the PyTorch of this interpreter."""
    import torch
    at = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(at, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-I{i}" for i in include], CALLS_SRC, "-o", out, f"-L{lib}", f"-Wl,-rpath,{lib}",
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"]


def _newer(out: str, sources) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(d) > os.path.getmtime(out) for d in sources)


def build_calls(force: bool = False) -> str:
    """Builds _calls.so when it is missing or older than its sources."""
    if force or _newer(CALLS_OUT, [CALLS_SRC, os.path.join(ROOT, "include", "sigattn.h")]):
        tmp = CALLS_OUT + ".tmp"
        subprocess.run(calls_cmd(tmp), check=True)
        os.replace(tmp, CALLS_OUT)
    return CALLS_OUT


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds libsigattn.so and _calls.so where they are missing or older than
    their sources; returns the library's path."""
    with ThreadPoolExecutor(1) as pool:
        calls = pool.submit(build_calls, force)
        _build_library(force, verbose)
        calls.result()
    return OUT


def _build_library(force: bool, verbose: bool) -> str:
    if not force and not _newer(OUT, DEPS):
        return OUT
    os.makedirs(OBJ, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else []
    newest_header = max(os.path.getmtime(h) for h in HEADERS)
    objs, todo = [], []
    for unit in UNITS:
        obj = os.path.join(OBJ, unit[:-3] + ".o")
        objs.append(obj)
        src = max(newest_header, os.path.getmtime(os.path.join(CSRC, unit)))
        if force or not os.path.exists(obj) or os.path.getmtime(obj) <= src:
            todo.append(compile_cmd(unit, obj, extra))
    with ThreadPoolExecutor(max(1, min(len(todo) or 1, os.cpu_count() or 1))) as pool:
        list(pool.map(lambda cmd: subprocess.run(cmd, check=True), todo))
    tmp = OUT + ".tmp"
    subprocess.run(link_cmd(objs, tmp), check=True)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force="-i" not in sys.argv, verbose="-v" in sys.argv))
