"""Builds libpa_b200.so, the sm_100a CUDA library behind include/pa.h, in-tree.

    python -m paged_kv_cache_372_b200.build [--force] [--verbose]

nvcc compiles each csrc/*.cu (with the kernel headers it includes) for sm_100a
only, side by side, and links the objects. Objects and library land in
``_lib/`` next to this file, so the library travels with the source tree; an
object is kept until its source or a header it includes is newer.
"""
from __future__ import annotations

import argparse
import glob
import hashlib
import os
import re
import shutil
import subprocess
import time
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(LIB_DIR, "libpa_b200.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa_b200")
    return path


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "pa.h")])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def includes(path: str) -> set[str]:
    """The source itself and the headers of this tree that it includes, in turn."""
    seen: set[str] = set()
    todo = [path]
    while todo:
        cur = todo.pop()
        if cur in seen:
            continue
        seen.add(cur)
        with open(cur) as f:
            names = re.findall(r'^\s*#include\s+"([^"]+)"', f.read(), flags=re.M)
        for name in names:
            for d in (CSRC, INCLUDE):
                if os.path.exists(os.path.join(d, name)):
                    todo.append(os.path.join(d, name))
    return seen


def _run(cmd: list[str], verbose: bool) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stdout + res.stderr)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None,
          out: str | None = None) -> str:
    """Compile when a source is newer than the library (or force). `extra` adds nvcc
    flags (e.g. -DPA_DECODE_STAGES=6); `out` writes the library elsewhere."""
    target = out or LIB
    if not force and out is None and not stale():
        return LIB
    os.makedirs(os.path.dirname(target), exist_ok=True)
    started = time.time()
    common = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE]
    if verbose:
        common.insert(1, "-Xptxas=-v")
    common += extra or []
    # Objects are kept per target and per set of flags.
    tag = "." + hashlib.sha256(" ".join(extra).encode()).hexdigest()[:8] if extra else ""
    objects, todo = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = f"{target}.{os.path.basename(src)[:-3]}{tag}.o"
        objects.append(obj)
        if force or verbose or not os.path.exists(obj) or any(
                os.path.getmtime(h) > os.path.getmtime(obj) for h in includes(src)):
            todo.append((src, obj))
    suffix = f".tmp{os.getpid()}"

    def compile_one(job: tuple[str, str]) -> None:
        src, obj = job
        begun = time.time()
        _run([*common, "-c", src, "-o", obj + suffix], verbose)
        os.utime(obj + suffix, (begun, begun))  # a source edited meanwhile is newer
        os.replace(obj + suffix, obj)

    with ThreadPoolExecutor(max_workers=max(1, min(len(todo), os.cpu_count() or 1))) as pool:
        list(pool.map(compile_one, todo))
    _run([nvcc(), *ARCH, "-shared", *objects, "-o", target + suffix], False)
    os.utime(target + suffix, (started, started))
    os.replace(target + suffix, target)
    return target


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
