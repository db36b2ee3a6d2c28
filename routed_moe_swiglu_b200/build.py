"""Build the CUDA library libroutedmoe.so in-tree with nvcc for sm_100a, and
_binding (for this interpreter), the short way from Python into it, with the
C++ compiler.

    python -m routed_moe_swiglu_b200.build [--force]

Every .cu under csrc/ is compiled (in parallel) with
``-gencode arch=compute_100a,code=sm_100a -lineinfo -O3`` and linked into
routed_moe_swiglu_b200/libroutedmoe.so; objects go to
routed_moe_swiglu_b200/_build/.  Only the CUDA runtime is linked; the
driver entry point for TMA descriptors is looked up at run time.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import sysconfig
from importlib.machinery import EXTENSION_SUFFIXES

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libroutedmoe.so")
# tagged: it uses the interpreter's full API, and another version must not load it
BINDING = os.path.join(PKG, "_binding" + EXTENSION_SUFFIXES[0])
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + os.path.join(ROOT, "include"),
         "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, extra, verbose):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, [src] + _headers() + [__file__]):
        cmd = [NVCC] + ARCH + FLAGS + extra + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
    return obj


def _build_binding(force, verbose):
    src, include = os.path.join(CSRC, "binding.cpp"), sysconfig.get_paths()["include"]
    untagged = os.path.join(PKG, "_binding.so")  # the name before: any interpreter would load it
    if os.path.exists(untagged):
        os.remove(untagged)
    if not (force or _stale(BINDING, [src] + _headers() + [__file__])):
        return
    why = None
    if not os.path.exists(os.path.join(include, "Python.h")):
        why = f"no {include}/Python.h"
    else:
        tmp = BINDING + ".tmp"
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + include,
               "-I" + os.path.join(ROOT, "include"), src, "-o", tmp]
        if verbose:
            print(" ".join(cmd), flush=True)
        try:
            subprocess.check_call(cmd)
            os.replace(tmp, BINDING)
        except (OSError, subprocess.CalledProcessError) as e:
            why = str(e)
    if why is not None:
        # the library does without it; one of other sources must not be loaded beside it
        if os.path.exists(BINDING):
            os.remove(BINDING)
        print(f"{why}: the compiled binding is not built, short calls go through ctypes", file=sys.stderr)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for f in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(f)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra, verbose), srcs))
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    _build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv))
