"""Build libsparse_act.so in-tree with hipcc for gfx950.

Usage: ``python -m sparse_input_gemv_amd.build`` (or ``build()`` from Python).
Every HIP source is compiled for gfx950 only; packed-fp32 instructions are
disabled for all device code.  Objects go to ``_build/`` at the repository
root, the shared library next to this file.
"""

from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsparse_act.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["sparsify.hip", "gemv.hip", "calibrate.hip", "gemm.hip", "stream.hip", "linear.hip",
           "grouped.hip", "grouped_backward.hip", "int8.hip", "abi.cpp", "validate.cpp"]
LINEAR_USERS = ["grouped.hip", "grouped_backward.hip", "int8.hip"]  # include linear.hip's tile engine

COMMON = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-I" + os.path.join(ROOT, "include")]
DEVICE = ["-x", "hip", "--offload-arch=gfx950",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def source_hash(src: str) -> str:
    """Of a source and every header it may include: an object's .src file
    holds the one it was built from."""
    inc = os.path.join(ROOT, "include")
    headers = [os.path.join(d, f) for d in (CSRC, inc) for f in sorted(os.listdir(d)) if f.endswith((".hpp", ".h"))]
    headers += [os.path.join(CSRC, "linear.hip")] if src in LINEAR_USERS else []
    h = hashlib.sha256()
    for path in [os.path.join(CSRC, src)] + headers:
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    if src.endswith(".hip"):
        cmd = [HIPCC] + DEVICE + COMMON + ["-c", path, "-o", obj]
    else:
        cmd = [HIPCC] + COMMON + ["-c", path, "-o", obj]
    built_from = source_hash(src)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    with open(obj + ".src", "w") as f:
        f.write(built_from)
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(SOURCES), int(os.environ.get("MAX_JOBS", "8")))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
