"""Build libleapquant.so (the sm_100a CUDA library behind include/leapquant.h)
in place, next to this file."""
from __future__ import annotations

import glob
import hashlib
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libleapquant.so")
OBJ = os.path.join(HERE, "_build")  # objects, one for each source

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
]


def _sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def _deps():
    return (_sources() + sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh")))
            + [os.path.join(ROOT, "include", "leapquant.h")])


def _built_with():
    """The additional flags the library was built with (none, where nothing says so)."""
    path = os.path.join(OBJ, "extra_flags")
    if not os.path.exists(path):
        return []
    with open(path) as f:
        return f.read().split("\n")[:-1]


def needs_build(extra=()) -> bool:
    if not os.path.exists(LIB) or _built_with() != list(extra):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _headers_of(src):
    """The csrc headers a source includes, directly or through others."""
    found, todo = set(), [src]
    while todo:
        for name in re.findall(r'^#include "(lq_\w+\.cuh)"', open(todo.pop()).read(), flags=re.M):
            path = os.path.join(HERE, "csrc", name)
            if path not in found:
                found.add(path)
                todo.append(path)
    return sorted(found) + [os.path.join(ROOT, "include", "leapquant.h"), os.path.abspath(__file__)]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile each source to an object (only those older than what they
    include, at once) and link them into libleapquant.so.  `extra`: more compiler
    flags; objects built with some are kept apart from those built without."""
    extra = list(extra)
    if not force and not needs_build(extra):
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    obj_dir = OBJ if not extra else os.path.join(OBJ, hashlib.sha256("\n".join(extra).encode()).hexdigest()[:16])
    os.makedirs(obj_dir, exist_ok=True)
    jobs, objs = [], []
    for src in _sources():
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if not force and os.path.exists(obj):
            t = os.path.getmtime(obj)
            if all(os.path.getmtime(p) <= t for p in [src, *_headers_of(src)]):
                continue
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", "-o", obj + ".tmp", src]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        jobs.append((cmd, obj, subprocess.Popen(cmd)))
    failed = [(cmd, p.returncode) for cmd, _, p in jobs if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(failed[0][1], failed[0][0])
    for _, obj, _ in jobs:
        os.replace(obj + ".tmp", obj)
    cmd = [nvcc, *NVCC_FLAGS, "-shared", "-o", LIB + ".tmp", *objs]
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    with open(os.path.join(OBJ, "extra_flags"), "w") as f:
        f.writelines(x + "\n" for x in extra)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
