"""Build libpa_b200.so (the C-ABI library) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import glob
import os
import re
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

# Kernels that must be launched with exactly so many registers a thread: their
# setmaxnreg split gives away and takes what the launch allots (kRegs of
# csrc/pa_prefill_i8.cuh).  Another compiler's choice fails the build, not the calls.
REGISTERS = {"prefill_i8_kernel": 80}


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(HERE, "..", "include", "pa.h")])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def check_registers(ptxas_log: str) -> int:
    """Reads what ptxas -v says; raises if a kernel of REGISTERS has another
    number.  Returns how many kernels it checked."""
    checked = 0
    for entry in ptxas_log.split("Compiling entry function '")[1:]:
        name = entry.split("'", 1)[0]
        for part, want in REGISTERS.items():
            if part not in name:
                continue
            used = re.search(r"Used (\d+) registers", entry)
            if used is None or int(used.group(1)) != want:
                raise RuntimeError(f"{name} has {used.group(1) if used else 'unknown'} registers, its register "
                                   f"split needs {want}")
            checked += 1
    return checked


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not stale():
        return LIB
    with tempfile.TemporaryDirectory() as tmp:
        running, objects = [], []
        for unit in UNITS:
            objects.append(os.path.join(tmp, unit + ".o"))
            cmd = [NVCC, "-Xptxas=-v", *FLAGS, *extra, "-c", os.path.join(CSRC, unit), "-o", objects[-1]]
            print(" ".join(cmd), file=sys.stderr)
            log = open(os.path.join(tmp, unit + ".log"), "w+")
            running.append((cmd, log, subprocess.Popen(cmd, stderr=log)))
        logs = ""
        for cmd, log, p in running:
            code = p.wait()
            log.seek(0)
            text = log.read()
            log.close()
            said = text if verbose or code != 0 else "\n".join(x for x in text.splitlines() if "warning" in x)
            if said:
                print(said, file=sys.stderr)
            if code != 0:
                for _, _, other in running:
                    other.wait()
                raise subprocess.CalledProcessError(code, cmd)
            logs += text
        if check_registers(logs) == 0:
            raise RuntimeError("the compiler's log names no kernel of " + ", ".join(REGISTERS))
        subprocess.run([NVCC, *FLAGS[:2], "-shared", *objects, "-o", LIB], check=True)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
