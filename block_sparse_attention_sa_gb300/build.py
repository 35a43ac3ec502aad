"""Builds libsa_gb300.so in-tree with nvcc for sm_103a (no cmake, no torch, no
Python headers), and the small Python module that marshals the paged-cache calls
to it.

    python -m block_sparse_attention_sa_gb300.build [--force] [--verbose-ptxas]

Each .cu is compiled to an object in parallel, then linked into a shared
library next to this file. The module (csrc/bind.cpp) reads torch's tensors
directly, so it is compiled against the torch and the Python that run this and
carries both in its name; where it does not compile, the library and all that
needs no module stand, and the paged-cache calls from Python say that it is
missing. Each part is rebuilt only when one of its sources is newer.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsa_gb300.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def module_path() -> str:
    """Where the module of this torch and this Python lies."""
    import torch

    return os.path.join(PKG, "_sa_bind.%s.torch-%s.so" % (
        sysconfig.get_config_var("SOABI"), torch.__version__))


def _older(built: str, deps) -> bool:
    if not os.path.exists(built):
        return True
    t = os.path.getmtime(built)
    return any(os.path.getmtime(p) > t for p in deps)


def _common():
    return [os.path.join(ROOT, "include", "sa.h"), os.path.abspath(__file__)]


def _library_stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _common())


def _module_stale() -> bool:
    return _older(module_path(), glob.glob(os.path.join(CSRC, "*.cpp")) + _common())


def _compile_module() -> None:
    import torch

    path = module_path()
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cmd = [shutil.which("g++") or "g++", "-shared", "-fPIC", "-O2", "-std=c++17",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-I", sysconfig.get_path("include"), "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), os.path.join(CSRC, "bind.cpp"),
           "-L", os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python",
           "-Wl,-rpath," + os.path.join(root, "lib"), "-o", path + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the binding does not compile:\n{r.stdout}\n{r.stderr}")
    os.replace(path + ".tmp", path)


def _compile_library(verbose_ptxas: bool = False) -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(ROOT, "include")]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, "-c", src, "-o", obj] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(sources())) as ex:
        results = list(ex.map(compile_one, sources()))
    if verbose_ptxas:
        for _, err in results:
            sys.stderr.write(err)
    tmp = LIB + ".tmp"
    cmd = [cc, "-shared", "-o", tmp] + [o for o, _ in results] + ARCH + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    with ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(_compile_module) if force or _module_stale() else None
        if force or _library_stale():
            _compile_library(verbose_ptxas)
        if module is not None:
            try:
                module.result()
            except (ImportError, OSError, RuntimeError) as e:
                sys.stderr.write(f"the module of the paged-cache calls was not built: {e}\n")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv))
