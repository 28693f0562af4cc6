"""Builds libsparseopt.so in-tree for GB300 (sm_103a) with nvcc.

Each translation unit under ``csrc/`` is compiled in parallel, then linked into
``lazy_optimizers_embedding_gb300/libsparseopt.so``; ``csrc/pycall.cpp`` becomes the
module ``_pycall.so`` (the binding's calls with tensors), against the library and the
installed PyTorch.  Objects go to ``_build/`` (git-ignored).  Rebuilds only when a
source or header is newer than the library.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsparseopt.so")
PYCALL_SRC = os.path.join(CSRC, "pycall.cpp")
PYCALL = os.path.join(PKG, "_pycall.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "-I", INCLUDE, "-I", CSRC]
# extra -D tuning defines (e.g. "-DSO_FUSED_MIN_BLOCKS=2"), for sweeps
EXTRA_DEFS = os.environ.get("SPARSEOPT_NVCC_DEFS", "").split()


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsparseopt")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


STAMP = os.path.join(BUILD, "defines.txt")   # the extra defines the current library was built with


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(PYCALL):
        return True
    try:
        with open(STAMP) as f:
            if f.read() != " ".join(EXTRA_DEFS):
                return True
    except OSError:
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(PYCALL))
    deps = [PYCALL_SRC] + sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *EXTRA_DEFS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    def compile_pycall():
        """The command that links the module, once the library is there."""
        import sysconfig

        import torch
        at = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(cc)))
        cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
        obj = os.path.join(BUILD, "pycall.cpp.o")
        cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
               "-isystem", os.path.join(at, "include"), "-isystem", sysconfig.get_paths()["include"],
               "-isystem", os.path.join(cuda, "include"), "-c", PYCALL_SRC, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cxx} failed on {PYCALL_SRC}:\n{r.stdout}\n{r.stderr}")
        return [cxx, "-shared", obj, "-L", PKG, "-l:libsparseopt.so", "-Wl,-rpath,$ORIGIN", "-L",
                os.path.join(at, "lib"),
                "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]

    srcs = sources()
    with ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        pycall = ex.submit(compile_pycall)
        objs = list(ex.map(compile_one, srcs))
        link_pycall = pycall.result()
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = PYCALL + f".{os.getpid()}.tmp"
    r = subprocess.run([*link_pycall, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, PYCALL)
    with open(STAMP, "w") as f:
        f.write(" ".join(EXTRA_DEFS))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
