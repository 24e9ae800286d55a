"""Builds libsigattn.so in-tree with nvcc for sm_100a (no GPU needed to build).

Every ``csrc/*.cu`` file is one translation unit; they compile side by side
into ``_build/`` and are linked into one library.  A unit is compiled again
when it or any header is newer than its object file."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
OUT = os.path.join(HERE, "libsigattn.so")
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


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds libsigattn.so when it is missing or older than its sources."""
    stale = force or not os.path.exists(OUT) or any(
        os.path.getmtime(d) > os.path.getmtime(OUT) for d in DEPS)
    if not stale:
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
