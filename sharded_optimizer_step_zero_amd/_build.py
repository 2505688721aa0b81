"""Compiles the product library libzeroshard.so in place (hipcc, gfx950)."""
from __future__ import annotations

import os
import subprocess
import tempfile

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(_HERE, "libzeroshard.so")
SOURCES = [os.path.join(_HERE, "csrc", f)
           for f in ("kernels.hip", "plan.cpp", "abi.cpp", "offload.cpp", "alloc.cpp",
                     "static_step.hip", "embed.hip", "norm.hip", "act8.hip", "xent.hip")]
# host-compiled part: the offloaded update (vector clones picked at load time)
HOST_SOURCES = [os.path.join(_HERE, "csrc", "host_step.cpp")]
GXX_FLAGS = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-fno-math-errno", "-pthread",
             "-Wall", "-Wextra"]

# -ffp-contract=off: no FMA contraction (each operation rounds once);
# correctly rounded fp32 division / sqrt; fp32 subnormals kept;
# packed-fp32 instructions disabled.
HIPCC_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
               "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
               "-fno-gpu-flush-denormals-to-zero",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Wall"]


def build(verbose: bool = False, extra_flags=None) -> str:
    with tempfile.TemporaryDirectory() as tmp:
        objs = []
        for src in HOST_SOURCES:
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            cmd = ["g++", *GXX_FLAGS, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
            objs.append(obj)
        # each source by itself, side by side (a file of kernels takes up to a minute)
        running = []
        for src in SOURCES:
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            cmd = ["hipcc", *HIPCC_FLAGS, *(extra_flags or []), "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append((cmd, subprocess.Popen(cmd)))
            objs.append(obj)
        # all of them end before the folder that they write to goes
        failed = [(cmd, p) for cmd, p in running if p.wait()]
        for cmd, p in failed:
            raise subprocess.CalledProcessError(p.returncode, cmd)
        # the objects go to the linker as they are (hipcc would read them as source)
        cmd = ["hipcc", *HIPCC_FLAGS, *(extra_flags or []), "-shared", "-o", LIB + ".tmp",
               *[f"-Wl,{o}" for o in objs], "-pthread"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB
