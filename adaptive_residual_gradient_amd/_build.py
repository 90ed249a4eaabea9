"""Build of the HIP library ``libadacomp.so`` for gfx950 with hipcc, and of the
operators' Python entry points (host code only) with g++."""
from __future__ import annotations

import os
import pathlib
import subprocess
import sysconfig

HERE = pathlib.Path(__file__).resolve().parent
SOURCES = [HERE / "csrc" / "adacomp.hip", HERE / "csrc" / "training.hip"]
LIB = HERE / "libadacomp.so"
BINDING = HERE / "_binding.so"

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # Bit-exact float32: no contraction of a*b+c into fused multiply-adds.
    "-ffp-contract=off",
    # No packed fp32 instructions (v_pk_add_f32 and friends).
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def build(verbose: bool = False) -> pathlib.Path:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB.with_suffix(".so.tmp")
    cmd = [hipcc, *HIPCC_FLAGS, "-o", str(tmp), *map(str, SOURCES)]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> pathlib.Path:
    """The extension module, against torch's headers and next to libadacomp.so."""
    import torch
    root = pathlib.Path(torch.__file__).resolve().parent
    tmp = BINDING.with_suffix(".so.tmp")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", str(root / "include"), "-isystem", str(root / "include/torch/csrc/api/include"),
           "-isystem", sysconfig.get_paths()["include"], "-o", str(tmp), str(HERE / "csrc" / "binding.cpp"),
           f"-L{HERE}", "-l:libadacomp.so", f"-L{root / 'lib'}", "-lc10", "-ltorch_cpu", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(verbose=True))
