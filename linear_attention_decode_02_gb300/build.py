"""Build libkda.so in-tree with nvcc for sm_103a (GB300), and with the C++ compiler
the small CPython module that marshals the binding's calls.

    python -m linear_attention_decode_02_gb300.build [--force] [--verbose]

Compiles each CUDA translation unit in parallel, then links one shared
library next to this file.  Rebuilds only when a source or header is newer
than the libraries.
"""

from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

import torch

from .binding import module_path

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda.so")
PYSRC = os.path.join(CSRC, "kda_python.cpp")
PYLIB = module_path(torch.__version__)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
              "-I", os.path.join(ROOT, "include")]


def _nvcc():
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkda")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [PYSRC, os.path.abspath(__file__)]


def up_to_date():
    if not (os.path.exists(LIB) and os.path.exists(PYLIB)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(PYLIB))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _compile(nvcc, src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc, *NVCC_FLAGS, *ARCH, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _python_module():
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no C++ compiler found for the binding's CPython module")
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    tmp = PYLIB + ".tmp"
    cmd = [cxx, "-std=c++17", "-O2", "-Wall", "-Wno-unknown-pragmas", "-fPIC", "-shared",
           "-isystem", os.path.join(home, "include"), "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
           PYSRC, "-o", tmp, "-L", os.path.join(home, "lib"), "-Wl,--no-as-needed", "-ltorch_python", "-ltorch_cuda",
           "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for {PYSRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, PYLIB)


def build(force=False, verbose=False):
    """Compile and link libkda.so; returns its path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        module = ex.submit(_python_module)
        results = list(ex.map(lambda s: _compile(nvcc, s, verbose), srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared", *ARCH, "-cudart", "shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    module.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
