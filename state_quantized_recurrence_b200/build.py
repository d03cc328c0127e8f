"""Build the CUDA library ``libgdn_qdq.so`` in-tree for sm_100a.

    python state_quantized_recurrence_b200/build.py [--force]

nvcc cross-compiles without a GPU.  Every ``csrc/*.cu`` is one object, the
objects are compiled side by side, and an object whose sources have not
changed is kept.  The shared library sits next to this file so that it
travels with the source tree.
"""

from __future__ import annotations

import concurrent.futures
import glob
import hashlib
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgdn_qdq.so")
OBJ = os.path.join(PKG, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-warn-spills",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


STAMP = LIB + ".sha256"


def _digest(paths) -> str:
    h = hashlib.sha256(" ".join(NVCC_FLAGS).encode())
    for s in paths:
        h.update(os.path.relpath(s, ROOT).encode())
        with open(s, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def source_digest() -> str:
    """Hash of the compiler flags and every source's name and contents.
    Staleness is decided by content, not modification times, which a copy
    of the tree to another machine need not preserve."""
    return _digest(_sources())


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(STAMP)):
        return False
    with open(STAMP) as f:
        return f.read().strip() == source_digest()


def _reached(path, seen=None):
    """`path` and every header of this library that it includes."""
    seen = [] if seen is None else seen
    if path in seen:
        return seen
    seen.append(path)
    with open(path) as f:
        names = re.findall(r'^\s*#include\s+"([^"]+)"', f.read(), flags=re.M)
    for n in names:
        for d in (CSRC, INCLUDE):
            p = os.path.join(d, n)
            if os.path.exists(p):
                _reached(p, seen)
    return seen


def _object(src, force, verbose) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    stamp = obj + ".sha256"
    digest = _digest(sorted(_reached(src)))
    if not force and os.path.exists(obj) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == digest:
                return obj
    flags = [f for f in NVCC_FLAGS if f != "-shared"]
    cmd = [_nvcc(), *flags, "-I", INCLUDE, "-c", "-o", obj + ".tmp", src]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(obj + ".tmp", obj)
    with open(stamp, "w") as f:
        f.write(digest + "\n")
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    digest = source_digest()
    os.makedirs(OBJ, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with concurrent.futures.ThreadPoolExecutor(max(1, min(8, len(sources)))) as pool:
        objects = list(pool.map(lambda s: _object(s, force, verbose), sources))
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *NVCC_FLAGS, "-o", tmp, *objects]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    with open(STAMP, "w") as f:
        f.write(digest + "\n")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
