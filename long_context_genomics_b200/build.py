"""Build libag.so (the CUDA kernels and the C ABI) in-tree for sm_100a, and
_layers.so (the compiled half of the layers' Python binding).

    python long_context_genomics_b200/build.py [--verbose] [--ptxas-v]

The library links the CUDA runtime statically and reaches the driver's
tensor-map encoder through cudaGetDriverEntryPoint, so it needs no CUDA
driver library at link time and cross-compiles on a machine without a GPU.
_layers.so is compiled by g++ against the headers of the installed torch and
works with that torch only: _layers.built_for names it, and another one builds
it anew.  Without torch the library is built alone (the C ABI needs nothing else).
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libag.so")
LAYERS = os.path.join(HERE, "_layers.so")
LAYERS_BUILT_FOR = os.path.join(HERE, "_layers.built_for")
LAYERS_SOURCE = os.path.join(CSRC, "layers_binding.cpp")
SOURCES = ["ag_api.cu", "ag_layers_api.cu", "attn_fwd_sm100.cu", "attn_noalloc.cu", "attn_bwd.cu",
           "attn_bwd_sm100.cu", "pair_bias_project.cu", "linear.cu", "linear_sm100.cu",
           "qk_norm_rope.cu", "grad_clip.cu"]
HEADERS = ["sm100.cuh", "ag_internal.h", "attn_bwd_phases.cuh", "linear_epilogue.cuh",
           "linear_gemm.h", "linear_ptx.cuh", "launch.cuh"]
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


def torch_dir():
    """Where torch is installed, or None (torch itself is not imported)."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def built_for(torch: str) -> str:
    """What a _layers.so depends on: the torch and the Python it is compiled for."""
    with open(os.path.join(torch, "version.py")) as f:
        version = re.search(r"__version__\s*=\s*['\"]([^'\"]+)", f.read())
    return f"torch {version.group(1) if version else '?'} {sysconfig.get_config_var('SOABI')}"


def _layers_stale() -> bool:
    torch = torch_dir()
    if torch is None:
        return False
    if _stale(LAYERS, [LAYERS_SOURCE, os.path.join(ROOT, "include", "ag.h")]):
        return True
    if not os.path.exists(LAYERS_BUILT_FOR):
        return True
    with open(LAYERS_BUILT_FOR) as f:
        return f.read().strip() != built_for(torch)


def needs_build() -> bool:
    return _stale(LIB, _inputs()) or _layers_stale()


def _layers_command(torch: str):
    # torch's own flag for the C++ library's ABI, asked of that torch.
    abi = subprocess.run([sys.executable, "-c", "import torch; print(int(torch.compiled_with_cxx11_abi()))"],
                         capture_output=True, text=True)
    if abi.returncode != 0:
        raise RuntimeError("_layers build failed: torch does not import:\n" + abi.stderr)
    cmd = [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi.stdout.strip()}",
           f'-DAG_BUILT_FOR="{built_for(torch)}"']
    for d in (os.path.join(torch, "include"),
              os.path.join(torch, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], os.path.join(CUDA, "include")):
        cmd += ["-I", d]
    return cmd + ["-o", LAYERS, LAYERS_SOURCE, "-L", os.path.join(torch, "lib"), "-lc10",
                  "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]


def _build_layers(torch: str, verbose: bool) -> None:
    cmd = _layers_command(torch)
    if verbose:
        print(" ".join(cmd))
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("_layers build failed:\n" + res.stdout + res.stderr)
    with open(LAYERS_BUILT_FOR, "w") as f:
        f.write(built_for(torch) + "\n")


def build(verbose: bool = False, ptxas_v: bool = False) -> str:
    """Builds both; a failure of _layers.so is raised when libag.so is done."""
    cmd = [
        NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-O3",
        "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-shared",
        "--expt-relaxed-constexpr", "--threads", "0", "-I", os.path.join(ROOT, "include"),
        "-o", LIB,
    ] + [os.path.join(CSRC, s) for s in SOURCES]
    if ptxas_v:
        cmd[1:1] = ["-Xptxas", "-v"]
    if verbose:
        print(" ".join(cmd))
    # (nvcc's output goes to a file, so that it never waits for a reader.)
    with tempfile.TemporaryFile("w+") as log:
        lib = subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT)
        torch, failed = torch_dir(), None
        try:
            if torch is None:
                print("torch is not installed: _layers.so (the layers' Python binding) is not built")
            else:
                _build_layers(torch, verbose)
        except (RuntimeError, OSError) as e:
            failed = e
        finally:
            lib.wait()
        log.seek(0)
        out = log.read()
    if lib.returncode != 0:
        raise RuntimeError("libag build failed:\n" + out)
    if verbose or ptxas_v:
        sys.stdout.write(out)
    if failed is not None:
        raise failed
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
