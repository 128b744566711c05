"""Build ``libhyena_conv.so`` (the C ABI of include/hyena_conv.h) for sm_100a with nvcc.

The library is built in-tree, next to this file.  ``python -m gated_causal_fir_b200.build``
or :func:`build` from Python.  Needs nvcc; cross-compiles on a host without a GPU.
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libhyena_conv.so")
INCLUDE = os.path.join(ROOT, "include")
SOURCES = [os.path.join(CSRC, f) for f in ("hyena_conv.cu", "hyena_scan.cu", "hyena_proj.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
    os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in DEPS)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if a source is newer than it (or force); return its path."""
    if not force and up_to_date():
        return LIB
    tmp = LIB + ".tmp%d" % os.getpid()

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    def compile_one(src):
        obj = "%s.%s.o" % (tmp, os.path.basename(src))
        run([nvcc()] + NVCC_FLAGS + ["-I", INCLUDE, "-c", src, "-o", obj])
        return obj

    try:
        with ThreadPoolExecutor(len(SOURCES)) as pool:  # one nvcc per source, side by side
            objs = list(pool.map(compile_one, SOURCES))
        run([nvcc()] + NVCC_FLAGS + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    finally:
        for src in SOURCES:
            obj = "%s.%s.o" % (tmp, os.path.basename(src))
            if os.path.exists(obj):
                os.remove(obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
