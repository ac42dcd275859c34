"""Build the CUDA library libdsaidx.so in-tree for sm_100a (B200).

Usage: python -m sparse_attention_token_dsa_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libdsaidx.so")
OBJ = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr"]


def units():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def sources():
    return sorted(units() + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "dsaidx.h")])


def _reads(path: str, seen=None) -> set:
    """A source file and the library's own headers that it includes."""
    seen = set() if seen is None else seen
    path = os.path.normpath(path)
    if path not in seen:
        seen.add(path)
        for name in re.findall(r'^#include "([^"]+)"', open(path).read(), flags=re.M):
            _reads(os.path.join(os.path.dirname(path), name), seen)
    return seen


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile each .cu that changed (all of them when forced), side by side, and
    link the library."""
    if not force and not stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    objects, running = [], []
    for u in units():
        obj = os.path.join(OBJ, os.path.basename(u)[:-3] + ".o")
        objects.append(obj)
        if force or not os.path.exists(obj) or any(
                os.path.getmtime(s) > os.path.getmtime(obj) for s in _reads(u)):
            tmp = obj + f".tmp{os.getpid()}.o"
            cmd = [NVCC, *FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-c", u, "-o", tmp]
            running.append((subprocess.Popen(cmd), cmd, tmp, obj))
    failed = None
    for p, cmd, tmp, obj in running:
        if p.wait() != 0:
            failed = failed or subprocess.CalledProcessError(p.returncode, cmd)
        else:
            os.replace(tmp, obj)
    if failed:
        raise failed
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, *FLAGS, "-shared", *objects, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
