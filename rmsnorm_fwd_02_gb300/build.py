"""Builds the CUDA library ``librmsnorm_train.so`` in-tree, for sm_103a only.

Each translation unit is compiled by its own nvcc process (in parallel), then nvcc
links the shared library with the static CUDA runtime.  No GPU is needed to build.
ptxas resource usage (registers, spills, shared memory) is written to
``_build/ptxas.log`` for inspection.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "librmsnorm_train.so")
SOURCES = ["rmsn_api.cu", "rmsn_fwd.cu", "rmsn_bwd.cu", "rmsn_bwd_rc.cu", "rmsn_small.cu",
           "rmsn_drop_fwd.cu", "rmsn_drop_bwd.cu", "drop.cu", "gn_api.cu",
           "gn_fwd.cu", "gn_bwd.cu", "ln_api.cu", "ln_fwd.cu", "ln_bwd.cu"]
HEADERS = ["rmsn_common.cuh", "rmsn_launch.h", "rmsn_fwd_rows.cuh", "rmsn_bwd_rows.cuh",
           "rmsn_tmem.cuh", "drop_launch.h", "drop_philox.cuh", "types.cuh", "gn_launch.h",
           "gn_common.cuh", "ln_launch.h",
           "ln_common.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build")
    return cand


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files += [os.path.join(ROOT, "include", h) for h in ("rmsnorm_train.h", "layernorm_train.h",
                                                    "dropout_train.h", "groupnorm_train.h")]
    return files


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles (if needed) and returns the path of ``librmsnorm_train.so``."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I", os.path.join(ROOT, "include"), "-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *common, "-c", os.path.join(CSRC, src), "-o", obj]
        p = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, p

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    log = []
    for src, _, p in results:
        log.append(f"==== {src}\n{p.stdout}{p.stderr}")
        if p.returncode != 0:
            sys.stderr.write(p.stdout + p.stderr)
            raise RuntimeError(f"nvcc failed on {src}")
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write("\n".join(log))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp] + [r[1] for r in results]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        sys.stderr.write(p.stdout + p.stderr)
        raise RuntimeError("nvcc link failed")
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
