"""Build libevoattn.so in-tree with nvcc for sm_100a.

    python -m triangle_biased_attention_b200.build [--force] [--verbose]

The library is a plain shared object with a C ABI (include/evo_attn.h); it
links the CUDA runtime statically and takes the driver's tensor-map encoder
through the runtime's entry-point query, so it needs no libcuda at link time.
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libevoattn.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
]

# translation units: attention and triangle multiplication; the transition and
# the relative-position bias
UNITS = ["evo_attn.cu", "evo_blocks.cu"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  [os.path.join(INCLUDE, "evo_attn.h")])


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not is_stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    objs = [f"{tmp}.{os.path.splitext(u)[0]}.o" for u in UNITS]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)

    try:
        with ThreadPoolExecutor(len(UNITS)) as pool:
            list(pool.map(lambda uo: run([_nvcc(), *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-I", CSRC, "-c",
                                          os.path.join(CSRC, uo[0]), "-o", uo[1]]), zip(UNITS, objs)))
        run([_nvcc(), *NVCC_FLAGS, "-shared", *objs, "-o", tmp])
        os.replace(tmp, LIB)
    finally:
        for path in (*objs, tmp):
            if os.path.exists(path):
                os.remove(path)
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills per kernel")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose, extra_flags=extra))


if __name__ == "__main__":
    main()
