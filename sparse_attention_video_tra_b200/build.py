"""Build the in-tree C-ABI library ``libtra_b200.so`` for sm_100a with nvcc.

    python -m sparse_attention_video_tra_b200.build [--force]

nvcc cross-compiles without a GPU.  The plan code (tra_plan.cpp) is compiled
with -ffp-contract=off so radius arithmetic keeps its two separate roundings.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libtra_b200.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
SOURCES = ["tra_api.cu", "tra_grad.cu", "tra_cache.cu", "tra_plan.cpp"]


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "tra.h"))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    flags = [*ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-ffp-contract=off,-fvisibility=hidden",
             "-I", os.path.join(ROOT, "include")]
    # one nvcc per source, all at once, then the link
    objs = [f"{tmp}.{s}.o" for s in SOURCES]
    cmds = [[nvcc, *flags, "-c", "-o", o, os.path.join(CSRC, s)] for s, o in zip(SOURCES, objs)]
    link = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    try:
        running = []
        for cmd in cmds:
            if verbose:
                print(" ".join(cmd))
            running.append(subprocess.Popen(cmd))
        for proc, cmd in zip(running, cmds):
            if proc.wait():
                for other in running:
                    other.wait()
                raise subprocess.CalledProcessError(proc.returncode, cmd)
        if verbose:
            print(" ".join(link))
        subprocess.run(link, check=True)
        os.replace(tmp, LIB)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
