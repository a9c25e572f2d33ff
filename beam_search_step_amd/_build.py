"""Compile libbeamstep.so and libbeamattn.so for gfx950 with hipcc, in the
package directory. libbeamattn.so links against libbeamstep.so beside it."""
from __future__ import annotations

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "beamstep.hip")
INC = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libbeamstep.so")
ATTN_SRC = os.path.join(HERE, "csrc", "beamattn.hip")
ATTN_LIB = os.path.join(HERE, "libbeamattn.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-fno-fast-math", "-Wall",
    # packed fp32 instructions stay off: the compiler must not form them
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _compile(src: str, lib: str, verbose: bool, extra=()) -> None:
    tmp = lib + ".tmp"
    cmd = [HIPCC, *FLAGS, "-I", INC, "-o", tmp, src, *extra]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, lib)


def build(verbose: bool = False) -> str:
    _compile(SRC, LIB, verbose)
    _compile(ATTN_SRC, ATTN_LIB, verbose, ("-L", HERE, "-lbeamstep", "-Wl,-rpath,$ORIGIN"))
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
