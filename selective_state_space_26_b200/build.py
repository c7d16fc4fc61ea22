"""Build the CUDA libraries in-tree for sm_100a with nvcc: libjamba_ssm.so
(the scan and the decode update), libjamba_ssm_proj.so (the projection that
feeds the scan), libjamba_ssm_gated.so (the gated linear recurrence) and
libjamba_ssm_serve.so (8-bit projections and the maps of a continuous batch)."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "jamba_ssm.cu")
LIB = os.path.join(PKG, "libjamba_ssm.so")
PROJ_SRC = os.path.join(PKG, "csrc", "jamba_ssm_proj.cu")
PROJ_LIB = os.path.join(PKG, "libjamba_ssm_proj.so")
GATED_SRC = os.path.join(PKG, "csrc", "jamba_ssm_gated.cu")
GATED_LIB = os.path.join(PKG, "libjamba_ssm_gated.so")
SERVE_SRC = os.path.join(PKG, "csrc", "jamba_ssm_serve.cu")
SERVE_LIB = os.path.join(PKG, "libjamba_ssm_serve.so")
ALL = ((SRC, LIB), (PROJ_SRC, PROJ_LIB), (GATED_SRC, GATED_LIB), (SERVE_SRC, SERVE_LIB))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def sources():
    d = os.path.join(PKG, "csrc")
    return [os.path.join(d, f) for f in sorted(os.listdir(d)) if f.endswith((".cu", ".cuh", ".h"))]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    inc = os.path.join(ROOT, "include")
    deps = sources() + [os.path.join(inc, h) for h in os.listdir(inc) if h.endswith(".h")]
    return all(os.path.getmtime(s) <= t for s in deps)


def _nvcc(src: str, out: str, verbose: bool) -> None:
    # Hidden visibility: each library keeps its own kernels and device status
    # word; only the extern "C" entry points marked for export are visible.
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo",
           "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-cudart", "static",
           "-I", os.path.join(ROOT, "include"), "-o", out, src]
    if out != LIB:
        cmd[cmd.index("-fPIC")] = "-fPIC,-fvisibility=hidden"
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)


def build(verbose: bool = False, force: bool = False) -> str:
    todo = [(src, out) for src, out in ALL if force or not up_to_date(out)]
    with ThreadPoolExecutor(len(ALL)) as pool:  # one nvcc each
        list(pool.map(lambda so: _nvcc(so[0], so[1], verbose), todo))
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, force=True)
    for _, lib in ALL:
        print(lib)
