"""Builds libkfac.so (the HIP kernels + C ABI) in-tree for gfx950 with hipcc, and
the _objectives extension (calls of the objectives on torch tensors).

Usage: python -m second_order_optimizer_amd.build [-v]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkfac.so")
EXT = os.path.join(PKG, "_objectives.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# -packed-fp32-ops off: plain fp32 vector code, no packed-fp32 instructions.
HIP_FLAGS = ["--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Wall", "-Werror=uninitialized", "-Wno-unused-function", "-I", os.path.join(ROOT, "include")]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops' is not a recognized feature" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{out}")
    if verbose and out.strip():
        print(out)


def _build_extension(verbose) -> None:
    """csrc/binding.cpp (host code only) against torch's and Python's headers."""
    import torch
    base = os.path.dirname(torch.__file__)
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    flags = ["-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__",
             "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               os.path.join(rocm, "include"), sysconfig.get_paths()["include"]]
    for d in include:
        flags += ["-isystem", d]
    libs = ["-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    tmp = EXT + ".tmp"
    _run([os.environ.get("CXX", "g++")] + flags + [os.path.join(CSRC, "binding.cpp"), "-o", tmp] + libs, verbose)
    os.replace(tmp, EXT)


def build(verbose: bool = False, jobs: int = 8) -> str:
    """Compiles every csrc/*.hip, links libkfac.so and builds the extension; returns the library's path."""
    os.makedirs(OBJ, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    objs = [os.path.join(OBJ, os.path.basename(s)[:-4] + ".o") for s in srcs]

    def cc(pair):
        s, o = pair
        _run([HIPCC] + HIP_FLAGS + ["-c", s, "-o", o], verbose)

    with ThreadPoolExecutor(max(1, min(jobs, len(srcs) + 1))) as ex:
        ext = ex.submit(_build_extension, verbose)
        list(ex.map(cc, zip(srcs, objs)))
        ext.result()
    tmp = LIB + ".tmp"
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs, verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
