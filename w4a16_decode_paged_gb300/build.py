"""Build the sm_103a shared library libw4a16_gb300.so in-tree (nvcc, no cmake).

Each .cu file under csrc/ is compiled in parallel with
``-gencode arch=compute_103a,code=sm_103a`` and linked into one shared
library with a plain C ABI (include/w4a16.h).  The output goes to
``w4a16_decode_paged_gb300/_build/``.  Beside it goes _w4a16_torch.<python>-
<torch version>.so, the argument marshalling of the short calls
(csrc/torch_args.cpp, g++ against torch's headers; it holds no kernel and is
given the library's entries by address).  The library does not need it: where
torch or its headers are missing, it is left out.
"""
from __future__ import annotations

import concurrent.futures as cf
import functools
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libw4a16_gb300.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


ARGS_SRC = os.path.join(CSRC, "torch_args.cpp")


@functools.lru_cache(maxsize=None)
def _torch():
    """(torch's folder, its version), without importing it; (None, None): no torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None, None
    folder = os.path.dirname(spec.origin)
    with open(os.path.join(folder, "version.py")) as f:
        return folder, re.search(r"__version__ = '([^']+)'", f.read()).group(1)


def args_lib():
    """The marshalling module's file, named for the interpreter and the torch
    whose ABI it has; None without torch."""
    folder, version = _torch()
    return folder and os.path.join(BUILD, f"_w4a16_torch.{sys.implementation.cache_tag}-{version}.so")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


TRACE_BUILD = os.path.join(HERE, "_build_trace")
TRACE_LIB = os.path.join(TRACE_BUILD, "libw4a16_gb300_trace.so")


def build_trace(force: bool = False) -> str:
    """Kernel-timeline build (-DW4A16_TRACE): a separate library that adds
    w4a16_trace_start / w4a16_trace_count; the product library is untouched."""
    # separately compiled device functions must fit the register budget of
    # the kernels that call them (the persistent kernel runs 512 threads)
    return build(force=force, extra_flags=["-DW4A16_TRACE", "-rdc=true", "-maxrregcount=128"], out=TRACE_LIB)


def build(force: bool = False, verbose: bool = False, extra_flags=None, out: str = None) -> str:
    lib = out or LIB
    bdir = os.path.dirname(lib)
    if not force and os.path.exists(lib) and all(os.path.getmtime(p) <= os.path.getmtime(lib) for p in _deps()):
        if lib == LIB:
            build_args()
        return lib
    os.makedirs(bdir, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src).replace(".cu", ".o"))
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(10, len(srcs) + 1)) as ex:
        args = ex.submit(build_args, force) if lib == LIB else None
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".tmp{os.getpid()}"
    rdc = ["-rdc=true"] if "-rdc=true" in flags else []
    cmd = [cc, *ARCH, *rdc, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if args is not None:
        args.result()  # (an error of its own comes behind the library)
    return lib


def build_args(force: bool = False):
    """The native argument marshalling (a CPython module, host code only); None
    where there is no torch or no headers of it to build against."""
    out, folder = args_lib(), _torch()[0]
    inc = [os.path.join(folder, "include", *sub) for sub in ((), ("torch", "csrc", "api", "include"))] if folder else []
    if not inc or not os.path.isdir(os.path.join(inc[0], "ATen")):
        sys.stderr.write("torch's headers are not here: calls are checked in Python, _w4a16_torch is not built\n")
        return None
    deps = [ARGS_SRC, os.path.join(INCLUDE, "w4a16.h")]
    if not force and os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps):
        return out
    os.makedirs(BUILD, exist_ok=True)
    inc.append(os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"))
    lib = os.path.join(folder, "lib")
    tmp = out + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", ARGS_SRC, "-o", tmp,
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], *[x for p in inc for x in ("-isystem", p)],
           "-L", lib, f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {ARGS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    force = "--force" in sys.argv
    verbose = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force=force or bool(extra), verbose=verbose or bool(extra), extra_flags=extra))
