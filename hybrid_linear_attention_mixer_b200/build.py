"""Build the sm_100a CUDA library in place (nvcc; no GPU needed to compile)."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libgdn_b200.so")
CSRC = os.path.join(HERE, "csrc")
# translation unit -> the headers only it includes; COMMON is included by both
UNITS = {"gdn.cu": ("conv.cuh", "intra.cuh", "scan.cuh", "norm.cuh", "decode.cuh", "cp.cuh", "fixup.cuh"),
         "serve.cu": ("quant.cuh", "block_norm.cuh", "gemm_i8.cuh", "beam.cuh", "reorder.cuh")}
COMMON = ("device.cuh", "gemm.cuh", "host.cuh")
SOURCES = [os.path.join(CSRC, f) for u, deps in UNITS.items() for f in (u, *deps)] + \
          [os.path.join(CSRC, f) for f in COMMON]
HEADERS = [os.path.join(ROOT, "include", "gdn.h")]
NVCC_FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
              "-Xcompiler", "-fPIC"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libgdn_b200.so next to this file if it is missing or out of date: the
    stale translation units at the same time, then the link."""
    if not (force or stale(LIB, SOURCES + HEADERS)):
        return LIB
    objs, running = [], []
    for unit, deps in UNITS.items():
        obj = os.path.join(HERE, "build", unit[:-3] + ".o")
        objs.append(obj)
        if force or stale(obj, [os.path.join(CSRC, f) for f in (unit, *deps, *COMMON)] + HEADERS):
            os.makedirs(os.path.dirname(obj), exist_ok=True)
            tmp = obj + ".tmp%d" % os.getpid()
            cmd = [nvcc(), *NVCC_FLAGS, "-I" + os.path.join(ROOT, "include"), "-c", "-o", tmp, os.path.join(CSRC, unit)]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd), file=sys.stderr)
            running.append((subprocess.Popen(cmd), cmd, tmp, obj))
    failed = [cmd for proc, cmd, _, _ in running if proc.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, _, tmp, obj in running:
        os.replace(tmp, obj)
    tmp = LIB + ".tmp%d" % os.getpid()
    subprocess.check_call([nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
