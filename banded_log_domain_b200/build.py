"""Builds libsinkhorn_attn.so in-tree with nvcc for sm_100a.

    python -m banded_log_domain_b200.build [--force]
"""
from __future__ import annotations

import glob
import json
import os
import subprocess
import sys
import time

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
OBJ = os.path.join(ROOT, "build")  # object files and how they were made, one folder per library
TMP = f".tmp{os.getpid()}"


def dep_list(dep_file: str):
    """The files that a compilation read, as nvcc listed them."""
    with open(dep_file) as f:
        return f.read().replace("\\\n", " ").split(":", 1)[1].split()


def current(target: str, record: str, cmd) -> bool:
    """Whether ``target`` was made by ``cmd`` from files that have not changed since:
    by what ``record`` says, which is written when the target is complete."""
    try:
        with open(record) as f:
            r = json.load(f)
        t = os.path.getmtime(target)
        return r["cmd"] == cmd and all(os.path.getmtime(f) <= t for f in r["files"])
    except (OSError, ValueError, KeyError):
        return False


def put(target: str, record: str, tmp: str, cmd, files, began: float):
    """``tmp`` becomes ``target``, as old as the command's start (a source written while
    it ran is newer), and the record says how it was made."""
    os.utime(tmp, (began, began))
    if os.path.exists(record):
        os.remove(record)
    os.replace(tmp, target)
    with open(record + TMP, "w") as f:
        json.dump({"cmd": cmd, "files": files}, f)
    os.replace(record + TMP, record)


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds the library and its bounds-checked debug twin (-DSA_DEBUG): the
    stale sources compiled side by side, then linked.  Everything is written under
    a name of this process and then renamed, so that a build that is killed, or
    another at the same time, leaves nothing half-written behind."""
    jobs, links = [], []
    for lib, extra, sub in ((LIB, [], "release"), (DEBUG_LIB, ["-DSA_DEBUG"], "debug")):
        out = os.path.join(OBJ, sub)
        os.makedirs(out, exist_ok=True)
        objs = []
        for src in sources():
            obj = os.path.join(out, os.path.splitext(os.path.basename(src))[0] + ".o")
            objs.append(obj)
            cmd = [NVCC, *FLAGS, *extra, "-c", src]
            if force or not current(obj, obj + ".json", cmd):
                run = cmd + ["-MD", "-MF", obj + ".d" + TMP, "-o", obj + TMP]
                if verbose:
                    print(" ".join(run), flush=True)
                jobs.append((cmd, obj, time.time(), subprocess.Popen(run)))
        links.append((lib, os.path.join(out, "link.json"), objs))
    for _, _, _, p in jobs:
        p.wait()
    failed = None
    for cmd, obj, began, p in jobs:
        if p.returncode == 0:
            put(obj, obj + ".json", obj + TMP, cmd, dep_list(obj + ".d" + TMP), began)
        else:
            failed = subprocess.CalledProcessError(p.returncode, cmd)
        for f in (obj + TMP, obj + ".d" + TMP):
            if os.path.exists(f):
                os.remove(f)
    if failed:
        raise failed
    for lib, record, objs in links:
        cmd = [NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs]
        if force or not current(lib, record, cmd):
            began = time.time()
            run = cmd + ["-o", lib + TMP]
            if verbose:
                print(" ".join(run), flush=True)
            subprocess.check_call(run)
            put(lib, record, lib + TMP, cmd, objs, began)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
