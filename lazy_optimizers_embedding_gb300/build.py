"""Builds libsparseopt.so in-tree for GB300 (sm_103a) with nvcc.

Each translation unit under ``csrc/`` is compiled in parallel, then linked into
``lazy_optimizers_embedding_gb300/libsparseopt.so``; ``csrc/pycall.cpp`` becomes the
module ``_pycall.so`` (the binding's calls with tensors), against the library and the
installed PyTorch.  Objects go to ``_build/`` (git-ignored).  Rebuilds only when a
source or header is newer than the library, and the module also for another Python or
PyTorch.  Where the module cannot be built (no C++ compiler, no headers) the library is
built all the same, and ctypes takes the module's calls.
"""
from __future__ import annotations

import glob
import os
import platform
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
PYCALL_STAMP = os.path.join(BUILD, "pycall.txt")   # the Python and PyTorch the module was built for


def pycall_key() -> str:
    """The Python and PyTorch that a module built now would be for."""
    import torch
    return f"{platform.machine()} {sys.implementation.cache_tag} torch {torch.__version__}"


def _read(path) -> str | None:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def pycall_usable() -> bool:
    """Whether the module is there and was built for this Python and PyTorch."""
    return os.path.exists(PYCALL) and _read(PYCALL_STAMP) == pycall_key()


def _older(path, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps)


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale() -> bool:
    return (_read(STAMP) != " ".join(EXTRA_DEFS) or
            _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers()))


def _pycall_stale() -> bool:
    deps = [PYCALL_SRC] + _headers()
    if _read(PYCALL_STAMP) == "none for " + pycall_key():   # it could not be built, and nothing has changed
        return _older(PYCALL_STAMP, deps)
    return not pycall_usable() or _older(PYCALL, deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    library, module = force or _stale(), force or _pycall_stale()
    if not library and not module:
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

    def link(cmd, to):
        tmp = to + f".{os.getpid()}.tmp"
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, to)

    srcs = sources() if library else []
    with ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        pycall = ex.submit(compile_pycall) if module else None
        objs = list(ex.map(compile_one, srcs))
    if library:
        link([cc, *ARCH, "-shared", *objs], LIB)
        with open(STAMP, "w") as f:
            f.write(" ".join(EXTRA_DEFS))
    if module:
        key = pycall_key()
        try:
            link(pycall.result(), PYCALL)
        except (RuntimeError, OSError) as e:   # the library is whole without it
            sys.stderr.write(f"no compiled calls (ctypes takes the operators' calls): {e}\n")
            key = "none for " + key
        with open(PYCALL_STAMP, "w") as f:
            f.write(key)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
