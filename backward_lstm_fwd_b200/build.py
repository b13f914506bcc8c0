"""Build liblstm.so in-tree for sm_100a with nvcc.

    python -m backward_lstm_fwd_b200.build [--force] [--verbose]

The library links the CUDA runtime statically and reaches driver-only entry
points (tensor-map encoding) through cudaGetDriverEntryPoint, so it loads on
machines without a GPU driver; only its compute calls need a device.
"""
from __future__ import annotations

import contextlib
import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_PATH = os.path.join(PKG, "liblstm.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return (sorted(glob.glob(os.path.join(CSRC, "*.cu")))
            + sorted(glob.glob(os.path.join(CSRC, "*.cuh")))
            + sorted(glob.glob(os.path.join(ROOT, "include", "*.h"))))


def _stale(out: str) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in _sources() + [__file__])


def _sweep(*dirs: str) -> None:
    """Remove what builds that were killed have left (their process is gone)."""
    for path in (f for d in dirs for f in glob.glob(os.path.join(d, "*.tmp[0-9]*"))):
        try:
            os.kill(int(re.search(r"\.tmp(\d+)", os.path.basename(path)).group(1)), 0)
        except ProcessLookupError:
            with contextlib.suppress(FileNotFoundError):  # (another build swept it)
                os.remove(path)
        except PermissionError:  # someone else's, and alive
            pass


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale(LIB_PATH):
        return LIB_PATH
    obj_dir = os.path.join(PKG, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    _sweep(obj_dir, PKG)
    flags = [_nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC,-O2,-Wall",
             "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags += ["-Xptxas", "-v"]
    headers = [s for s in _sources() if not s.endswith(".cu")] + [__file__]
    objs, jobs = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):  # one object each, side by side
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if not force and os.path.exists(obj) and all(
                os.path.getmtime(s) <= os.path.getmtime(obj) for s in headers + [src]):
            continue
        tmp = obj + f".tmp{os.getpid()}.o"
        jobs.append((subprocess.Popen([*flags, "-c", "-o", tmp, src]), tmp, obj, src))
    lib_tmp = LIB_PATH + f".tmp{os.getpid()}"
    try:
        failed = [src for p, _, _, src in jobs if p.wait() != 0]
        if failed:
            raise RuntimeError(f"nvcc failed on {', '.join(failed)}")
        for _, tmp, obj, _ in jobs:
            os.replace(tmp, obj)
        subprocess.run([*flags, "-shared", "-o", lib_tmp, *objs], check=True)
        os.replace(lib_tmp, LIB_PATH)
    finally:  # of a failed or interrupted build nothing goes on or stays
        for p, _, _, _ in jobs:
            if p.poll() is None:
                p.terminate()
                p.wait()
        for tmp in [lib_tmp, *(tmp for _, tmp, _, _ in jobs)]:
            if os.path.exists(tmp):
                os.remove(tmp)
    return LIB_PATH


if __name__ == "__main__":
    p = build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(p)
