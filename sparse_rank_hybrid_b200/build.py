"""Build libslra.so in-tree with nvcc for sm_100a (cross-compiles without a GPU)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libslra.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def deps() -> list[str]:
    return sources() + sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh"))) + [os.path.join(ROOT, "include", "slra.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    # the files side by side, then one link: the row kernels' many types would otherwise double the build
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
             "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", os.path.join(ROOT, "include"),
             "-Xptxas", "-v" if verbose else "-O3"]
    with tempfile.TemporaryDirectory(prefix="libslra") as objects:
        def compile_one(src: str):
            obj = os.path.join(objects, os.path.basename(src) + ".o")
            return obj, subprocess.run([NVCC, *flags, "-c", src, "-o", obj], capture_output=True, text=True)

        with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
            done = list(pool.map(compile_one, sources()))
        _check([r for _, r in done], verbose)
        tmp = LIB + f".tmp{os.getpid()}"
        _check([subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp,
                                *(obj for obj, _ in done)], capture_output=True, text=True)], False)
        os.replace(tmp, LIB)
    return LIB


def _check(runs, verbose: bool) -> None:
    for r in runs:
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc failed building libslra.so")
        if verbose:
            sys.stderr.write(r.stderr)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
