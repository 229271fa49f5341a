"""Build the HIP libraries (libspecverify.so, libspecforward.so) in-tree for gfx950."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "spec_verify.hip")
FORWARD_SRC = os.path.join(HERE, "csrc", "spec_forward.hip")
INC = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libspecverify.so")
FORWARD_LIB = os.path.join(HERE, "libspecforward.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Werror",
    "-Wno-unused-command-line-argument",
]


def build(verbose: bool = False) -> str:
    """Compile both libraries (at the same time); the path of libspecverify.so."""
    jobs = []
    for src, lib in ((SRC, LIB), (FORWARD_SRC, FORWARD_LIB)):
        cmd = [HIPCC, *FLAGS, "-I", INC, "-o", lib + ".tmp", src]
        if verbose:
            print(" ".join(cmd), flush=True)
        jobs.append((lib, cmd, subprocess.Popen(cmd)))
    failed = [subprocess.CalledProcessError(p.returncode, cmd) for _, cmd, p in jobs if p.wait() != 0]
    if failed:
        raise failed[0]
    for lib, _, _ in jobs:
        os.replace(lib + ".tmp", lib)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
