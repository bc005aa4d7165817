"""Builds libforge_attn.so (the CUDA library behind include/) and _front.so (the torch front
end of the operators around the attention, a CPython module over it) in-tree.

    python -m causal_attention_fwd_attn_b200.build [--verbose]

nvcc compiles for sm_100a only (tcgen05 and TMA need the arch-specific target);
no GPU is needed to build.  ``--ptxas-info`` adds ``-Xptxas -v`` (registers,
spills and shared memory per kernel).

The library needs nvcc alone (run this file itself where torch is missing); without torch, or its
headers or Python's, the front end is left out and the build says so.
"""
from __future__ import annotations

import argparse
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libforge_attn.so")
FRONT = os.path.join(PKG, "_front.so")
FRONT_SOURCE = os.path.join(CSRC, "front.cpp")
SOURCES = ["forge_attn_api.cu", "attn_fwd.cu", "attn_bwd.cu", "tc_probe.cu", "forge_attn_noalloc.cu",
           "adamw.cu", "gemm.cu", "convert.cu", "qkv.cu", "gemm_grouped.cu", "grad.cu"]
HEADERS = ["sm100_ptx.cuh", "sm100_grouped_ptx.cuh", "forge_internal.h"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    return [os.path.join(INCLUDE, h) for h in ("forge_attn.h", "forge_attn_testing.h", "forge_adamw.h",
                                               "forge_linear.h")]


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    return files + _headers()


def _newer(target, files) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in files)


def front_lacks():
    """What is missing to build the front end, None if nothing is."""
    import sysconfig

    try:
        import torch
    except ImportError:
        return "torch"
    root = os.path.dirname(os.path.abspath(torch.__file__))
    for what, path in (("torch's headers", os.path.join(root, "include", "ATen", "ATen.h")),
                       ("torch with CUDA", os.path.join(root, "lib", "libc10_cuda.so")),
                       ("Python's headers", os.path.join(sysconfig.get_paths()["include"], "Python.h"))):
        if not os.path.exists(path):
            return f"{what} ({path})"
    return None if shutil.which("g++") else "g++"


def front_tag() -> str:
    """What the front end depends on beside its sources: it is compiled against the headers, and
    so the object layouts, of one torch and one Python."""
    import sysconfig

    import torch

    return (f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"Python {sysconfig.get_config_var('EXT_SUFFIX')}")


def front_built_for():
    """The tag that the built front end carries, without loading it; None if there is none."""
    if not os.path.exists(FRONT):
        return None
    with open(FRONT, "rb") as f:
        found = re.search(rb"forge front end built for ([^\0]*)\0", f.read())
    return found.group(1).decode() if found else None


def _front_current() -> bool:
    return _newer(FRONT, [FRONT_SOURCE] + _headers()) and front_built_for() == front_tag()


def up_to_date() -> bool:
    return _newer(LIBRARY, _inputs()) and (front_lacks() is not None or _front_current())


def _build_front(verbose: bool) -> None:
    """Compiles csrc/front.cpp against the headers of the torch that runs it and links it with
    the library beside it."""
    import sysconfig

    import torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    includes = [os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"],
                os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")]
    cmd = [shutil.which("g++"), "-std=c++17", "-O2", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DFORGE_FRONT_TAG="{front_tag()}"', "-I", INCLUDE]
    for p in includes:
        cmd += ["-isystem", p]
    cmd += [FRONT_SOURCE, "-o", FRONT + ".tmp", "-L", PKG, "-l:" + os.path.basename(LIBRARY),
            "-Wl,-rpath,$ORIGIN", "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python"]
    _run(cmd, "g++", verbose)
    os.replace(FRONT + ".tmp", FRONT)


def _run(cmd, what, verbose, show=False) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{what} failed")
    if show or verbose:
        sys.stderr.write(res.stderr)


def build(force: bool = False, ptxas_info: bool = False, verbose: bool = False) -> str:
    if not force and not ptxas_info and up_to_date():
        return LIBRARY
    # No relocatable device code: ptxas then honours per-warpgroup register budgets
    # (setmaxnreg), which the dK/dV kernel relies on.
    cmd = [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared",
           "-Xcompiler", "-fPIC", "-I", INCLUDE, "-o", LIBRARY + ".tmp"]
    if ptxas_info:
        cmd += ["-Xptxas", "-v"]
    cmd += [os.path.join(CSRC, s) for s in SOURCES]
    if force or ptxas_info or not _newer(LIBRARY, _inputs()):
        _run(cmd, "nvcc", verbose, show=ptxas_info)
        os.replace(LIBRARY + ".tmp", LIBRARY)
    lacks = front_lacks()
    if lacks is not None:
        sys.stderr.write(f"{os.path.basename(FRONT)} is not built: no {lacks}\n")
    elif force or not _front_current():
        _build_front(verbose)
    return LIBRARY


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    a = ap.parse_args()
    print(build(force=True, ptxas_info=a.ptxas_info, verbose=a.verbose))


if __name__ == "__main__":
    main()
