"""Build libattn_gb300.so in-tree with nvcc for sm_103a (no cmake, no torch extension).

Each CUDA translation unit compiles in parallel to ``_build/*.o``; the objects link into
``exact_io_aware_09_gb300/libattn_gb300.so`` with the CUDA runtime linked statically.
Usage: ``python exact_io_aware_09_gb300/build.py [-v] [--force]`` (the package itself cannot be
imported before the library exists).
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libattn_gb300.so")
SOURCES = ["attn_api.cu", "attn_fwd.cu", "attn_fwd_paged.cu", "attn_paged_few.cu", "attn_fwd_window.cu", "attn_fwd_pair.cu",
           "attn_decode.cu", "attn_decode_fp8.cu", "attn_cache_fp8.cu", "attn_pages.cu", "attn_cache_fp4.cu", "attn_paged_fp4.cu", "attn_paged_fp4_chunk.cu",
           "attn_bwd.cu", "attn_bwd_window.cu", "attn_fp8.cu"]
HEADERS = [os.path.join(CSRC, h)
           for h in ("ptx.cuh", "internal.h", "attn_fwd_two.cuh", "attn_decode.cuh",
                     "attn_rows.cuh", "attn_bwd.cuh", "attn_cache.cuh", "attn_paged.cuh",
                     "fp4.cuh")] + [
    os.path.join(ROOT, "include", "attn.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + HEADERS):
            cmd = [nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose else []) + [
                "-c", s, "-o", o]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)

    if jobs:
        with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
