"""Builds the CUDA library in-tree: ``_lib/libgdn_gb300.so`` for sm_103a.

Two translation units (``csrc/gdn_api.cu`` and ``csrc/gdn_recurrent.cu``, which include the
kernels), compiled side by side, so a build takes about half a minute on either the x86 build
host or the Arm GPU host.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
UNITS = ("gdn_api", "gdn_recurrent")
OUT_DIR = os.path.join(HERE, "_lib")
OUT = os.path.join(OUT_DIR, "libgdn_gb300.so")

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return [f for pattern in ("csrc/*.cu", "csrc/*.cuh", "csrc/*.h") for f in glob.glob(os.path.join(HERE, pattern))] + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    if not force and os.path.exists(OUT):
        newest = max(os.path.getmtime(d) for d in sources())
        if os.path.getmtime(OUT) >= newest:
            return OUT
    tmp = OUT + f".tmp{os.getpid()}"
    extra = ["-Xptxas=-v"] if verbose else []
    objects = [f"{tmp}.{u}.o" for u in UNITS]
    jobs = [subprocess.Popen([nvcc(), *extra, *NVCC_FLAGS, "-c", "-o", o, os.path.join(HERE, "csrc", u + ".cu")])
            for u, o in zip(UNITS, objects)]
    codes = [j.wait() for j in jobs]
    try:
        for job, code in zip(jobs, codes):
            if code:
                raise subprocess.CalledProcessError(code, job.args)
        subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objects], check=True)
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force=True, verbose=True))
