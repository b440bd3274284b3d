"""Build libzero.so, the CUDA library behind the binding, for sm_103a, and
_calls, the CPython module that marshals its most frequent calls.

Each translation unit is compiled in parallel with nvcc, then linked into a
shared library next to this file (in-tree, so the binding finds it).  No
fast-math and no flush-to-zero: the step's numerics are defined operation by
operation, and -fmad=false keeps any multiply-add from being fused.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libzero.so")
# named for the interpreter, so that another one does not load it
CALLS = os.path.join(HERE, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["zero_abi.cu", "zero_step_kernels.cu", "zero_gather.cu", "zero_advance.cu",
           "zero_embed.cu", "zero_dropout.cu", "zero_mx4.cu", "zero_mx4_matmul.cu",
           "zero_ops_abi.cu"]
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
HEADERS = ["zero_internal.h", "zero_ops.h", "zero_row_copy.cuh", "zero_elems.cuh", os.path.join("..", "..", "include", "zero.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "-fmad=false", "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
              "-Xcompiler", "-Wall"] + ARCH


def _newest_input() -> float:
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.abspath(__file__)]
    return max(os.path.getmtime(p) for p in paths)


def build_calls(force: bool = False) -> str:
    """The CPython module of csrc/zero_calls.c (host code only).  Without the
    interpreter's headers it is left out: the training operators then raise where
    they are called, and everything else works."""
    src = os.path.join(CSRC, "zero_calls.c")
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(INCLUDE, "zero.h"),
                                               os.path.abspath(__file__)))
    if not force and os.path.exists(CALLS) and os.path.getmtime(CALLS) >= newest:
        return CALLS
    headers = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(headers, "Python.h")):
        print("no Python.h under %s: %s is not built" % (headers, os.path.basename(CALLS)),
              file=sys.stderr)
        return CALLS
    tmp = CALLS + ".tmp.%d" % os.getpid()
    subprocess.run(["gcc", "-O2", "-std=c11", "-Wall", "-fPIC", "-shared", "-I", INCLUDE,
                    "-I", headers, src, "-o", tmp], check=True)
    os.replace(tmp, CALLS)
    return CALLS


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    build_calls(force)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = ["nvcc", *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp.%d" % os.getpid()
    subprocess.run(["nvcc", "-shared", *ARCH, "-cudart", "static", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
