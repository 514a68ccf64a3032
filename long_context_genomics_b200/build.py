"""Build libag.so (the CUDA kernels and the C ABI) in-tree for sm_100a, and
_layers.so (the compiled half of the layers' Python binding).

    python long_context_genomics_b200/build.py [--verbose] [--ptxas-v]

The library links the CUDA runtime statically and reaches the driver's
tensor-map encoder through cudaGetDriverEntryPoint, so it needs no CUDA
driver library at link time and cross-compiles on a machine without a GPU.
_layers.so is compiled by g++ against the headers of the installed torch.
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libag.so")
LAYERS = os.path.join(HERE, "_layers.so")
LAYERS_SOURCE = os.path.join(CSRC, "layers_binding.cpp")
SOURCES = ["ag_api.cu", "ag_layers_api.cu", "attn_fwd_sm100.cu", "attn_noalloc.cu", "attn_bwd.cu",
           "attn_bwd_sm100.cu", "pair_bias_project.cu", "linear.cu", "linear_sm100.cu",
           "qk_norm_rope.cu", "grad_clip.cu"]
HEADERS = ["sm100.cuh", "ag_internal.h", "attn_bwd_phases.cuh", "linear_epilogue.cuh",
           "linear_gemm.h", "launch.cuh"]
CUDA = "/usr/local/cuda"
NVCC = os.environ.get("NVCC", os.path.join(CUDA, "bin", "nvcc"))
CXX = os.environ.get("CXX", "g++")


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES + HEADERS]
            + [os.path.join(ROOT, "include", "ag.h")])


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in inputs)


def needs_build() -> bool:
    return (_stale(LIB, _inputs())
            or _stale(LAYERS, [LAYERS_SOURCE, os.path.join(ROOT, "include", "ag.h")]))


def _layers_command():
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cmd = [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden"]
    for d in (os.path.join(torch, "include"),
              os.path.join(torch, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], os.path.join(CUDA, "include")):
        cmd += ["-I", d]
    return cmd + ["-o", LAYERS, LAYERS_SOURCE, "-L", os.path.join(torch, "lib"), "-lc10",
                  "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]


def build(verbose: bool = False, ptxas_v: bool = False) -> str:
    cmd = [
        NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-O3",
        "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-shared",
        "--expt-relaxed-constexpr", "--threads", "0", "-I", os.path.join(ROOT, "include"),
        "-o", LIB,
    ] + [os.path.join(CSRC, s) for s in SOURCES]
    if ptxas_v:
        cmd[1:1] = ["-Xptxas", "-v"]
    layers = _layers_command()
    if verbose:
        print(" ".join(cmd))
        print(" ".join(layers))
    other = subprocess.Popen(layers, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    other_out, _ = other.communicate()
    if res.returncode != 0:
        raise RuntimeError("libag build failed:\n" + res.stdout + res.stderr)
    if other.returncode != 0:
        raise RuntimeError("_layers build failed:\n" + other_out)
    if verbose or ptxas_v:
        sys.stdout.write(res.stdout + res.stderr)
    return LIB


def ensure_built() -> str:
    if needs_build():
        build()
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true")
    a = ap.parse_args()
    print(build(verbose=a.verbose, ptxas_v=a.ptxas_v))
