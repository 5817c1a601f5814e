"""Build the C-ABI library ``libindexcache.so`` in-tree with nvcc for sm_100a.

Usage: ``python -m lightning_indexer_cross_b200.build [--force]``. Objects go
to ``_build/`` at the repository root; the shared library is written next to
this file so the Python binding finds it.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
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


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "indexcache.h"))
    return files


def needs_build() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(FRONT):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(FRONT))
    return any(os.path.getmtime(f) > t for f in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
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
    build_front(cc)
    return LIB


def build_front(cc: str) -> None:
    """The tensor front end, a Python extension that links the library (and torch's, which are loaded with torch)."""
    import torch
    root = os.path.dirname(torch.__file__)
    include = os.path.join(root, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
    lib = os.path.join(root, "lib")
    tmp = FRONT + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-fPIC", "-O2", "-std=c++17", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", include, "-isystem",
           os.path.join(include, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", cuda, os.path.join(CSRC, "front.cpp"), "-o", tmp, "-L", PKG, "-l:libindexcache.so", "-L", lib,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on front.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FRONT)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))
