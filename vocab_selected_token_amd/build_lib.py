"""Build step for librlk_logp.so (hipcc, gfx950 only).

Run ``python vocab_selected_token_amd/build_lib.py`` (or ``__graft_entry__.build()``).
The library is built in-tree so that it travels with the source tree.
"""
from __future__ import annotations

import os
import subprocess
import sys
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
LIB = PKG / "librlk_logp.so"
CALIB = PKG / "rlk_calib"  # stream-ceiling probe the benchmark reports beside its rates
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

HIP_SOURCES = ["rlk_kernels", "rlk_lmhead", "rlk_lmhead_bwd", "rlk_fp8",
               "rlk_noalloc", "rlk_process", "rlk_linear"]

# -ffp-contract=off: only the explicit fmaf calls fuse, so every tile's
# arithmetic is fixed by the source.  Packed fp32 VALU ops are disabled.
HIP_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
             "-ffp-contract=off", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def build() -> Path:
    """Compile the kernels (HIP, gfx950) and the boundary (host C++) and link the library;
    also build the stream-ceiling probe rlk_calib."""
    obj_dir = PKG / "_build"
    obj_dir.mkdir(exist_ok=True)
    inc = [f"-I{ROOT / 'include'}", f"-I{CSRC}"]
    b_obj = obj_dir / "rlk_boundary.o"
    hip_objs = [obj_dir / f"{name}.o" for name in HIP_SOURCES]
    for name, obj in zip(HIP_SOURCES, hip_objs):
        subprocess.run([HIPCC, *HIP_FLAGS, *inc, "-c", str(CSRC / f"{name}.hip"),
                        "-o", str(obj)], check=True)
    subprocess.run([HIPCC, "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__",
                    "-I/opt/rocm/include", *inc, "-c", str(CSRC / "rlk_boundary.cpp"),
                    "-o", str(b_obj)], check=True)
    tmp = LIB.with_name(LIB.name + ".tmp")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC",
                    *map(str, hip_objs), str(b_obj), "-o", str(tmp)], check=True)
    os.replace(tmp, LIB)
    tmp = CALIB.with_name(CALIB.name + ".tmp")
    subprocess.run([HIPCC, *HIP_FLAGS, str(CSRC / "rlk_calib.hip"), "-o", str(tmp)], check=True)
    os.replace(tmp, CALIB)
    return LIB


if __name__ == "__main__":
    print(build())
    sys.exit(0)
