"""Build the C-ABI library ``libindexcache.so`` in-tree with nvcc for sm_100a,
and ``_front.so``, the tensor front end of the paged latent cache, for the torch
and the Python that run this.

Usage: ``python -m lightning_indexer_cross_b200.build [--force]``. Objects go
to ``_build/`` at the repository root; the shared libraries are written next to
this file so the Python binding finds them. The library needs nvcc alone; where
torch, Python's headers or a C++ compiler are missing it is built without the
front end, and a line on stderr says so.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libindexcache.so")
FRONT = os.path.join(PKG, "_front.so")
FRONT_FOR = os.path.join(BUILD, "front.txt")  # the torch and the Python that FRONT is bound to
FRONT_SOURCE = "front.cpp"
SOURCES = ["api.cu", "indexer.cu", "topk.cu", "sparse_mla.cu", "topk_noalloc.cu", "append.cu", "gate.cu", "context_parallel.cu", "topk_threshold.cu", "overlap.cu",
           "rope.cu", "latent_cache.cu", "latent_attention.cu", "latent_pair.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-diag-suppress", "177", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libindexcache.so")


def _stale(target: str, sources) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in sources)


def _header() -> str:
    return os.path.join(INCLUDE, "indexcache.h")


def lib_stale() -> bool:
    return _stale(LIB, [_header()] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != FRONT_SOURCE])


def front_missing() -> str:
    """What the front end's build lacks here; empty if nothing."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    if shutil.which(_cxx()) is None:
        return f"the C++ compiler {_cxx()}"
    return ""


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def _front_for() -> str:
    """The torch and the Python of this process: an extension is bound to both. (A torch that runs from its sources
    names no version here; ops.py compares the one that the extension was compiled for.)"""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "from source"
    return f"torch {version}, {sys.implementation.cache_tag}"


def front_stale() -> bool:
    if _stale(FRONT, [_header(), os.path.join(CSRC, FRONT_SOURCE)]) or not os.path.exists(FRONT_FOR):
        return True
    with open(FRONT_FOR) as f:
        return f.read() != _front_for()


def needs_build() -> bool:
    return lib_stale() or (not front_missing() and front_stale())


def build(force: bool = False, verbose: bool = False) -> str:
    if force or lib_stale():
        build_lib(verbose)
    missing = front_missing()
    if missing:
        if not os.path.exists(FRONT):
            print(f"_front.so is not built: {missing} is missing (ops.rope and ops.latent_* need it; libindexcache.so "
                  "and the other operators do not)", file=sys.stderr)
    elif force or front_stale():
        build_front(nvcc())
    return LIB


def build_lib(verbose: bool = False) -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, err in results:
            sys.stderr.write(err)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build_front(cc: str) -> None:
    """The tensor front end, a Python extension that links the library (and torch's, which are loaded with torch)."""
    import torch
    root = os.path.dirname(torch.__file__)
    include = os.path.join(root, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
    lib = os.path.join(root, "lib")
    os.makedirs(BUILD, exist_ok=True)
    tmp = FRONT + ".tmp"
    cmd = [_cxx(), "-shared", "-fPIC", "-O2", "-std=c++17", "-Wall", f'-DIC_TORCH_VERSION="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", include, "-isystem",
           os.path.join(include, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", cuda, os.path.join(CSRC, FRONT_SOURCE), "-o", tmp, "-L", PKG, "-l:libindexcache.so", "-L", lib,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on front.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FRONT)
    with open(FRONT_FOR, "w") as f:
        f.write(_front_for())


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))
