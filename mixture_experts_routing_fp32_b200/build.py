"""Builds libmoe.so (all CUDA kernels + the C ABI) in-tree for sm_100a: one
object per csrc/*.cu, compiled side by side, and one link.

    python -m mixture_experts_routing_fp32_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libmoe.so")
OBJ_DIR = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-I", os.path.join(ROOT, "include"),
    "--expt-relaxed-constexpr",
]


def units():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps(path, seen=None):
    """`path` and the repository's headers that it includes, directly or not."""
    seen = set() if seen is None else seen
    path = os.path.normpath(path)
    if path in seen or not os.path.exists(path):
        return seen
    seen.add(path)
    with open(path, encoding="utf-8") as f:
        for name in re.findall(r'^\s*#include "([^"]+)"', f.read(), flags=re.M):
            _deps(os.path.join(os.path.dirname(path), name), seen)
    return seen


def sources():
    return sorted(set().union(*(_deps(u) for u in units())))


def _older(target, files) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in files)


def stale() -> bool:
    return _older(OUT, sources())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not stale():
        return OUT
    os.makedirs(OBJ_DIR, exist_ok=True)
    running, objects, errors = [], [], []
    for u in units():
        obj = os.path.join(OBJ_DIR, os.path.basename(u)[:-3] + ".o")
        objects.append(obj)
        if not force and not _older(obj, _deps(u)):
            continue
        tmp = obj + ".%d.tmp.o" % os.getpid()
        cmd = [NVCC, *(f for f in FLAGS if f != "-shared"), *extra, "-c", u, "-o", tmp]
        if verbose:
            print(" ".join(cmd), flush=True)
        p = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        running.append((p, tmp, obj))
    for p, tmp, obj in running:
        said = p.communicate()[0]
        if p.returncode != 0:
            errors.append(said)
            continue
        if verbose and said:
            sys.stderr.write(said)
        os.replace(tmp, obj)
    if not errors:
        tmp = OUT + ".%d.tmp" % os.getpid()
        cmd = [NVCC, *FLAGS, *objects, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(tmp, OUT)
            return OUT
        errors.append(r.stdout + r.stderr)
    sys.stderr.write("".join(errors))
    raise RuntimeError("nvcc failed building libmoe.so")


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else [])
    print(OUT)
