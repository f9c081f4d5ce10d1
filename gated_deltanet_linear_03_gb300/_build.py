"""Build libgdn.so (sm_103a) in-tree with nvcc.

Each ``csrc/*.cu`` file is compiled to an object in parallel, then the objects
are linked into ``gated_deltanet_linear_03_gb300/libgdn.so``.  Rebuilds only
when a source or header is newer than the library.

``csrc/fast_calls.cpp`` is the Python binding's part in C++ (``_fast.so``, against
the installed torch); g++ compiles it beside the kernels.

``build(debug=True)`` makes the bounds-checking variant ``libgdn_debug.so``
(``-DGDN_DEBUG_BOUNDS``: the recurrence's kernels, chunked.cu, scan.cu and
decode.cu, check every computed global address and tensor-copy coordinate before
use; see csrc/gdn_internal.cuh).  It has the same ABI and is built only on
request.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libgdn_debug.so")
FAST_SRC = os.path.join(CSRC, "fast_calls.cpp")
FAST = os.path.join(PKG, "_fast.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libgdn")
    return path


def _inputs():
    return (glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build_fast(force: bool = False) -> str:
    """The binding's C++ module, compiled against the torch that is installed here."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inputs = (FAST_SRC, os.path.join(ROOT, "include", "gdn.h"), os.path.abspath(__file__), torch.version.__file__)
    if not force and os.path.exists(FAST) and all(os.path.getmtime(f) <= os.path.getmtime(FAST) for f in inputs):
        return FAST
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = FAST + f".{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(root, "include"), "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I" + cuda,
           "-I" + sysconfig.get_paths()["include"], FAST_SRC, "-o", tmp, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on fast_calls.cpp:\n{r.stderr}")
    os.replace(tmp, FAST)
    return FAST


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    lib, bdir = (LIB_DEBUG, BUILD_DEBUG) if debug else (LIB, BUILD)
    fast = None if debug else cf.ThreadPoolExecutor(max_workers=1).submit(build_fast, force)
    if not force and up_to_date(lib):
        if fast:
            fast.result()
        return lib
    os.makedirs(bdir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    cc = nvcc()
    extra = ["-DGDN_DEBUG_BOUNDS"] if debug else []

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose:
        for _, log in results:
            print(log)
    tmp = lib + f".{os.getpid()}.tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    if fast:
        fast.result()
    return lib


if __name__ == "__main__":  # pragma: no cover
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
