"""Build libexl3.so (sm_100a) in-tree with nvcc, and the compiled part of the
Python binding with the C compiler.

    python -m gemm_exl3_gemv_b200.build [--force]

The shared libraries land next to this file; the binding loads them from
there.  nvcc cross-compiles, so no GPU is needed to build.  The compiled part
of the binding is of one Python (its file name says which) and optional: where
there is no C compiler or no Python header it is left out, and the binding's
calls take 1 to 3 us longer.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libexl3.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++20", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "exl3.h")]


# The debug-bounds variant: every product kernel (trellis and 4-bit) checks the
# index of each access to the packed words, the workspace and the outputs,
# records a failed check in the workspace status word and skips the access (no
# trap).  The cache's and the attention's kernels check page and sequence numbers
# in every build and have no further checks in this one.
LIB_DEBUG = os.path.join(HERE, "libexl3_debug.so")


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in _inputs())


# object files, one per source and variant (git-ignored)
OBJ_DIR = os.path.join(HERE, "_build")


def _compile(lib: str, extra, verbose: bool):
    """Compile every source whose object is older than it or any header, side
    by side, and link the shared library."""
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    tag = os.path.splitext(os.path.basename(lib))[0]
    os.makedirs(OBJ_DIR, exist_ok=True)
    headers = [p for p in _inputs() + [os.path.abspath(__file__)] if not p.endswith(".cu")]
    newest = max(os.path.getmtime(p) for p in headers)
    flags = [*ARCH, *FLAGS, *extra, "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags.append("-Xptxas=-v")

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, f"{tag}_{os.path.splitext(os.path.basename(src))[0]}.o")
        if verbose or not os.path.exists(obj) or os.path.getmtime(obj) < max(newest, os.path.getmtime(src)):
            tmp = f"{obj}.tmp{os.getpid()}"
            cmd = [nvcc, *flags, "-c", "-o", tmp, src]
            if verbose:
                print(" ".join(cmd))
            subprocess.run(cmd, check=True)
            os.replace(tmp, obj)
        return obj

    with concurrent.futures.ThreadPoolExecutor(os.cpu_count()) as pool:
        objects = list(pool.map(compile_one, sources()))
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objects], check=True)
    os.replace(tmp, lib)


# the compiled part of the binding: calls that a decode step makes many times
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_SRC = os.path.join(CSRC, "binding.c")


def _compile_binding(force: bool):
    inputs = [BINDING_SRC, os.path.join(ROOT, "include", "exl3.h")]
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= max(map(os.path.getmtime, inputs)):
        return
    cc, headers = os.environ.get("CC", "gcc"), sysconfig.get_paths()["include"]
    if not shutil.which(cc) or not os.path.exists(os.path.join(headers, "Python.h")):
        print(f"no {cc}, or no Python.h in {headers}: the compiled binding is left out", file=sys.stderr)
        return
    tmp = f"{BINDING}.tmp{os.getpid()}"
    subprocess.run([cc, "-O2", "-Wall", "-fPIC", "-shared", "-I", headers, "-I", os.path.join(ROOT, "include"), "-o", tmp,
                    BINDING_SRC], check=True)
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False, debug: bool = True) -> str:
    """Build libexl3.so (and, unless debug=False, libexl3_debug.so) if stale."""
    _compile_binding(force)
    if force or stale(LIB):
        _compile(LIB, [], verbose)
    if debug and (force or stale(LIB_DEBUG)):
        _compile(LIB_DEBUG, ["-DEXL3_DEBUG_BOUNDS"], verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
