"""Builds libdflash2.so (the C ABI of include/dflash2.h) for sm_103a, in-tree.

Each CUDA translation unit is compiled in parallel with
`nvcc -gencode arch=compute_103a,code=sm_103a -lineinfo -O3`, then linked with
`nvcc -shared`.  Output: block_drafter_pos_gb300/_build/libdflash2.so.
Run as `python -m block_drafter_pos_gb300.builder [--verbose]`.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libdflash2.so")
ROOT = os.path.dirname(HERE)

SOURCES = ["api.cu", "gemv.cu", "wide.cu", "glue.cu", "attention.cu", "lmhead.cu", "select.cu", "verify.cu", "noalloc.cu",
           "paged_api.cu", "paged_cache.cu", "paged_attention.cu",
           "paged_chunk.cu", "sample.cu", "paged_prefix.cu", "pages_api.cu", "pages.cu", "rope.cu"]
# Compiled a second time with the flag, for attention over shared prefixes (paged_sched.cuh).
SHARED_SOURCES = ["paged_attention.cu", "paged_chunk.cu"]
SHARED_FLAG = "-DDF2_SHARED_PREFIX=1"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _flags(verbose: bool):
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                "-I", os.path.join(ROOT, "include")]
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def build(verbose: bool = False, force: bool = False) -> str:
    """Compiles and links; returns the library path.  Rebuilds only when a source or
    header is newer than the library (or force)."""
    os.makedirs(OUT_DIR, exist_ok=True)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "dflash2.h")]
    if not force and os.path.exists(LIB):
        t = os.path.getmtime(LIB)
        if all(os.path.getmtime(d) <= t for d in deps):
            return LIB
    nvcc = nvcc_path()
    flags = _flags(verbose)

    def compile_one(job):
        src, extra = job
        obj = os.path.join(OUT_DIR, src.replace(".cu", "_shared.o" if extra else ".o"))
        cmd = [nvcc] + flags + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    jobs = [(src, []) for src in SOURCES] + [(src, [SHARED_FLAG]) for src in SHARED_SOURCES]
    with ThreadPoolExecutor(len(jobs)) as ex:
        results = list(ex.map(compile_one, jobs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force=True))
