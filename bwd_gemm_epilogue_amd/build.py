"""Build the gfx950 HIP library ``libswiglu_mlp.so`` in-tree with hipcc, and
the native half of the binding, ``_host.so``, with the host compiler.

Usage: ``python -m bwd_gemm_epilogue_amd.build`` (or ``build()`` from
Python).  Always recompiles.  Extra hipcc flags may be appended with the
environment variable ``SWIGLU_HIPCC_FLAGS`` (diagnostics only).
"""
from __future__ import annotations

import concurrent.futures
import os
import shlex
import subprocess
import sys
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libswiglu_mlp.so")
HOST = os.path.join(PKG, "_host.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # identical fp32 rounding in every kernel that computes h: no implicit
    # contraction of a*b+c into fma (explicit fmaf only)
    "-ffp-contract=off",
    # never emit packed fp32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


SOURCES = ["swiglu_mlp.hip", "layer_norm.hip", "grad_clip.hip", "moe_few.hip"]


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = (r.stdout or "") + (r.stderr or "")
    # the host pass does not know the packed-fp32 target feature; that note is harmless
    lines = [l for l in out.splitlines() if "packed-fp32-ops" not in l]
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed:\n" + "\n".join(lines))
    if verbose and lines:
        print("\n".join(lines))


def _host_flags():
    """Include and link paths of Python and of torch's host libraries."""
    import torch
    at = os.path.dirname(torch.__file__)
    include = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    compile_ = ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *(f"-I{d}" for d in include)]
    link = [f"-L{os.path.join(at, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10",
            f"-L{PKG}", f"-l:{os.path.basename(LIB)}", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def build(verbose: bool = False) -> str:
    """Compile every source (in parallel) and link the library and the module."""
    extra = shlex.split(os.environ.get("SWIGLU_HIPCC_FLAGS", ""))
    host_compile, host_link = _host_flags()
    with tempfile.TemporaryDirectory() as tmp, concurrent.futures.ThreadPoolExecutor() as pool:
        objs = [os.path.join(tmp, s + ".o") for s in SOURCES]
        host_obj = os.path.join(tmp, "host.o")
        jobs = [pool.submit(_run, [HIPCC, *FLAGS, "-c", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                                   os.path.join(CSRC, s), "-o", o, *extra], verbose) for s, o in zip(SOURCES, objs)]
        jobs.append(pool.submit(_run, [CXX, *host_compile, "-c", os.path.join(CSRC, "host.cpp"), "-o", host_obj], verbose))
        for j in jobs:
            j.result()
        _run([HIPCC, *FLAGS, "-shared", *objs, "-o", LIB + ".tmp", *extra], verbose)
        os.replace(LIB + ".tmp", LIB)
        _run([CXX, "-shared", host_obj, "-o", HOST + ".tmp", *host_link], verbose)
        os.replace(HOST + ".tmp", HOST)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
