"""Build libfa_gb300.so in-tree with nvcc for sm_103a, and tensor_calls.so with the host compiler (no cmake).

    python exact_tiled_attention_26_gb300/build.py [--verbose] [--ptxas-info]

Each translation unit compiles in parallel into ``_build/``; the objects are
linked (static CUDA runtime) into ``exact_tiled_attention_26_gb300/libfa_gb300.so``,
which knows nothing of PyTorch.  ``tensor_calls.so`` beside it is a Python module on
PyTorch's C++ tensors that calls the library; without PyTorch it is left out.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfa_gb300.so")
CALLS = os.path.join(PKG, "tensor_calls.so")
SOURCES = ["api.cu", "fwd.cu", "fwd_pp.cu", "fwd_persist.cu", "bwd.cu", "bwd_tile.cu", "bwd_persist.cu", "bwd2k.cu", "aux.cu", "bwd_noalloc.cu", "host_step.cu",
           "norm_rope.cu", "cache.cu", "fwd_tree.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libfa_gb300.so")


def _calls_cmd(nvcc):
    """The compile command of tensor_calls.cpp (PyTorch is found, not imported) and its link command; None without
    PyTorch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = os.path.dirname(spec.origin)
    includes = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
                os.path.join(torch, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
                os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
    obj = os.path.join(BUILD, "tensor_calls.o")
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f'-DFA_PACKAGE="{os.path.basename(PKG)}"', *[a for d in includes for a in ("-isystem", d)],
                "-c", os.path.join(CSRC, "tensor_calls.cpp"), "-o", obj]
    link = ["g++", "-shared", obj, "-o", CALLS + ".tmp", "-L", PKG, "-l:libfa_gb300.so", "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return compile_, link


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    p = subprocess.run(cmd, capture_output=True, text=True)
    if verbose and (p.stdout or p.stderr):
        print(p.stdout + p.stderr, flush=True)
    if p.returncode != 0:
        raise RuntimeError(f"command failed ({p.returncode}): {' '.join(cmd)}\n{p.stdout}\n{p.stderr}")
    return p.stdout + p.stderr


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    jobs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        jobs.append((obj, [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]))
    calls_cmd = _calls_cmd(nvcc)
    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        calls = ex.submit(_run, calls_cmd[0], verbose) if calls_cmd else None
        logs = list(ex.map(lambda j: _run(j[1], verbose), jobs))
    tmp = LIB + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *[j[0] for j in jobs]], verbose)
    os.replace(tmp, LIB)
    if calls_cmd:  # after the library, which does not depend on it
        calls.result()
        _run(calls_cmd[1], verbose)
        os.replace(CALLS + ".tmp", CALLS)
    else:
        print("PyTorch is not installed: tensor_calls.so is not built", file=sys.stderr)
    if ptxas_info:
        print("\n".join(logs))
    return LIB


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB)
