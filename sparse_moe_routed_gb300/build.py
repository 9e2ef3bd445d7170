"""Build libmoe.so and libmoe_block.so (the CUDA kernels + C ABIs) in-tree for
sm_103a.

Each translation unit compiles in parallel with nvcc, then the shared libraries
are linked next to this file.  No cmake, no torch extension machinery: the
libraries have plain C ABIs (include/moe.h, include/moe_block.h) and are loaded
with ctypes.  Loading one library builds that one alone.
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


def _sources(lib):
    return sources() if lib == LIB else block_sources()


def _deps(lib):
    """Files that `lib` is made of.  libmoe_block includes headers of csrc/, libmoe none of csrc_block/."""
    own = [CSRC] if lib == LIB else [CSRC_BLOCK, CSRC]
    headers = [f for d in own for ext in ("*.cuh", "*.h") for f in glob.glob(os.path.join(d, ext))]
    public = [os.path.join(INCLUDE, "moe.h")] + ([] if lib == LIB else [os.path.join(INCLUDE, "moe_block.h")])
    return _sources(lib) + headers + public


def up_to_date(lib: str | None = None) -> bool:
    """Is `lib` (None: both libraries) newer than everything that it is made of?"""
    return all(os.path.exists(f) and all(os.path.getmtime(d) <= os.path.getmtime(f) for d in _deps(f))
               for f in ((LIB, LIB_BLOCK) if lib is None else (lib,)))


def build(force: bool = False, verbose: bool = False, extra_flags=None, lib: str | None = None) -> str:
    """Build `lib`, LIB or LIB_BLOCK (None: both), where it is out of date; returns its path (None: libmoe.so's)."""
    stale = [f for f in ((LIB, LIB_BLOCK) if lib is None else (lib,)) if force or not up_to_date(f)]
    if not stale:
        return lib or LIB
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

    todo = [src for f in stale for src in _sources(f)]
    with ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 4)) as ex:
        objs = dict(zip(todo, ex.map(compile_one, todo)))
    for f in stale:
        tmp = f + ".tmp"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *(objs[s] for s in _sources(f)), "-lcudart_static", "-ldl", "-lrt",
             "-lpthread"], "link failed")
        os.replace(tmp, f)
    return lib or LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
