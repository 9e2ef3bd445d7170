"""Build libmoe.so and libmoe_block.so (the CUDA kernels + C ABIs) in-tree for
sm_103a.

Each translation unit compiles in parallel with nvcc, then the shared libraries
are linked next to this file.  No cmake, no torch extension machinery: the
libraries have plain C ABIs (include/moe.h, include/moe_block.h) and are loaded
with ctypes.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmoe.so")
CSRC_BLOCK = os.path.join(HERE, "csrc_block")
LIB_BLOCK = os.path.join(HERE, "libmoe_block.so")
BUILD_DIR = os.path.join(HERE, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def block_sources():
    return sorted(glob.glob(os.path.join(CSRC_BLOCK, "*.cu")))


def _deps():
    return [f for d in (CSRC, CSRC_BLOCK, INCLUDE) for ext in ("*.cu", "*.cuh", "*.h")
            for f in glob.glob(os.path.join(d, ext))]


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(LIB_BLOCK)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(LIB_BLOCK))
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Build both libraries; returns the path of libmoe.so."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)

    def compile_one(src):
        name = os.path.basename(src)
        obj = os.path.join(BUILD_DIR, os.path.basename(os.path.dirname(src)) + "_" + name + ".o")
        run([nvcc, *ARCH, *flags, "-c", src, "-o", obj], f"nvcc failed on {name}")
        return obj

    libs = ((LIB, sources()), (LIB_BLOCK, block_sources()))
    with ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 4)) as ex:
        objs = dict(zip((src for _, srcs in libs for src in srcs),
                        ex.map(compile_one, (src for _, srcs in libs for src in srcs))))
    for lib, srcs in libs:
        tmp = lib + ".tmp"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *(objs[s] for s in srcs), "-lcudart_static", "-ldl", "-lrt",
             "-lpthread"], "link failed")
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
