"""Build libpa_b200.so (the C-ABI library) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpa_b200.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
]

# translation units, compiled side by side
UNITS = ("pa_api.cu", "pa_serving.cu")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(HERE, "..", "include", "pa.h")])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not stale():
        return LIB
    with tempfile.TemporaryDirectory() as tmp:
        running, objects = [], []
        for unit in UNITS:
            objects.append(os.path.join(tmp, unit + ".o"))
            cmd = [NVCC, *FLAGS, *extra, "-c", os.path.join(CSRC, unit), "-o", objects[-1]]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
            running.append((cmd, subprocess.Popen(cmd)))
        failed = [(cmd, p.returncode) for cmd, p in running if p.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(failed[0][1], failed[0][0])
        subprocess.run([NVCC, *FLAGS[:2], "-shared", *objects, "-o", LIB], check=True)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
