"""Builds libsinkhorn_attn.so in-tree with nvcc for sm_100a.

    python -m banded_log_domain_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libsinkhorn_attn.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


DEBUG_LIB = os.path.join(PKG, "libsinkhorn_attn_debug.so")
OBJ = os.path.join(ROOT, "build")  # object files and their dependency lists, one folder per library


def deps(dep_file: str):
    """The files an object was compiled from, as nvcc listed them (None: never compiled)."""
    if not os.path.exists(dep_file):
        return None
    with open(dep_file) as f:
        return f.read().replace("\\\n", " ").split(":", 1)[1].split()


def stale(target: str, files) -> bool:
    if files is None or not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(not os.path.exists(f) or os.path.getmtime(f) > t for f in files)


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds the library and its bounds-checked debug twin (-DSA_DEBUG): the
    stale sources compiled side by side, then linked."""
    jobs, links = [], []
    for lib, extra, sub in ((LIB, [], "release"), (DEBUG_LIB, ["-DSA_DEBUG"], "debug")):
        out = os.path.join(OBJ, sub)
        os.makedirs(out, exist_ok=True)
        objs = []
        for src in sources():
            obj = os.path.join(out, os.path.splitext(os.path.basename(src))[0] + ".o")
            objs.append(obj)
            if force or stale(obj, deps(obj + ".d")):
                cmd = [NVCC, *FLAGS, *extra, "-c", "-MD", "-MF", obj + ".d", "-o", obj, src]
                if verbose:
                    print(" ".join(cmd), flush=True)
                jobs.append((cmd, obj, subprocess.Popen(cmd)))
        links.append((lib, objs))
    failed = [obj for _, obj, p in jobs if p.wait() != 0]
    for obj in failed:  # nothing half-written is taken for current
        if os.path.exists(obj):
            os.remove(obj)
    for cmd, obj, p in jobs:
        if p.returncode != 0:
            raise subprocess.CalledProcessError(p.returncode, cmd)
    for lib, objs in links:
        if force or stale(lib, objs):
            tmp = lib + f".tmp{os.getpid()}"
            cmd = [NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.check_call(cmd)
            os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
