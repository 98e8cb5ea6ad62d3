"""Build the CUDA library in-tree: decode_step_kv_gb300/_build/libfa_decode.so.

A few translation units compiled side by side, one -gencode (sm_103a), static
CUDA runtime.  Used by ``__graft_entry__.build()`` and by the binding on first use.
"""
from __future__ import annotations

import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SRCS = [os.path.join(CSRC, f) for f in ("fa_decode.cu", "fa_int4.cu", "fa_evict.cu",
                                         "fa_rope.cu", "fa_prefill.cu")]
HDRS = [os.path.join(ROOT, "include", "fa_decode.h"), os.path.join(CSRC, "fa_common.cuh")]
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libfa_decode.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return cand


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in (*SRCS, *HDRS, __file__))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = LIB + f".tmp{os.getpid()}"
    objs, running = [], []
    for src in SRCS:
        obj = os.path.join(OUT_DIR, os.path.basename(src) + f".{os.getpid()}.o")
        cmd = [nvcc(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-c",
               "-o", obj, src]
        if verbose:
            cmd.insert(2, "-Xptxas=-v")
        objs.append(obj)
        running.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE,
                                        text=True))
    done = [p.communicate() for p in running]
    try:
        for p, (_, err) in zip(running, done):
            if p.returncode != 0:
                raise RuntimeError(f"nvcc failed ({p.returncode}):\n{err}")
            if verbose:
                print(err)
        res = subprocess.run([nvcc(), ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs],
                             capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc link failed ({res.returncode}):\n{res.stderr}")
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
