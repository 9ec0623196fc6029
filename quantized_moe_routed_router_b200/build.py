"""Builds the CUDA library ``libts_moe.so`` in-tree for sm_100a with nvcc.

``python -m quantized_moe_routed_router_b200.build`` (or ``build()``) compiles
``csrc/ts_moe.cu`` and ``csrc/ops/ops.cu`` when the library is missing or older
than any source.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OPS = os.path.join(CSRC, "ops")
OBJ = os.path.join(PKG, "_build")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libts_moe.so")
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17", "-Xcompiler",
              "-fPIC", "--expt-relaxed-constexpr"]


def _files(*dirs) -> list:
    return sorted(p for d in dirs for e in ("*.cu", "*.cuh", "*.h") for p in glob.glob(os.path.join(d, e)))


def sources() -> list:
    return _files(CSRC, OPS, INCLUDE)


def units() -> list:
    """(source, object, files it is built from) of each translation unit."""
    base = _files(CSRC, INCLUDE)
    return [(os.path.join(CSRC, "ts_moe.cu"), os.path.join(OBJ, "ts_moe.o"), base),
            (os.path.join(OPS, "ops.cu"), os.path.join(OBJ, "ops.o"), base + _files(OPS))]


def _fresh(target: str, files: list) -> bool:
    return os.path.exists(target) and os.path.getmtime(target) >= max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and _fresh(LIB, sources()):
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    os.makedirs(OBJ, exist_ok=True)
    jobs, objs = [], []
    for src, obj, files in units():
        objs.append(obj)
        if force or not _fresh(obj, files):
            tmp = obj + f".tmp{os.getpid()}.o"
            cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", tmp]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd), file=sys.stderr)
            jobs.append((subprocess.Popen(cmd), cmd, tmp, obj))
    failed = None
    for p, cmd, tmp, obj in jobs:
        if p.wait():
            failed = subprocess.CalledProcessError(p.returncode, cmd)
        else:
            os.replace(tmp, obj)
    if failed:
        raise failed
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, *NVCC_FLAGS, "-shared", *objs, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
