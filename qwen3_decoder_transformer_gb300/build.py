"""Build the CUDA library in-tree: qwen3_decoder_transformer_gb300/_build/libqwen3_gb300.so.

Each translation unit in csrc/ is compiled by nvcc for sm_103a only (one -gencode) in parallel,
then linked into one shared library with the CUDA runtime linked statically. No CMake. Beside it, tensors.cpp
(the binding's checks of tensors for the paged and packed operators) becomes an extension module, one for each PyTorch and
Python. The library does not need it: where it cannot be compiled, build() warns, and those operators raise.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libqwen3_gb300.so")
SOURCES = ["gemm.cu", "kernels.cu", "attention.cu", "attention_tiles.cu", "attention_ranges.cu",
           "attention_packed.cu", "attention_paged4.cu", "paged4.cu", "logprobs.cu", "runtime.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return path


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "qwen3.h")]
    return max(os.path.getmtime(f) for f in files)


def tensors_path() -> str:
    """The extension module for the PyTorch and Python that run: it reads PyTorch's objects inline and is linked to where
    PyTorch's libraries are."""
    import torch

    made_for = "\n".join([torch.__version__, os.path.dirname(torch.__file__), sysconfig.get_config_var("EXT_SUFFIX") or ""])
    return os.path.join(BUILD, f"_tensors-{hashlib.sha256(made_for.encode()).hexdigest()[:12]}.so")


def _build_tensors() -> None:
    import torch

    root = os.path.dirname(torch.__file__)
    paths = [os.path.join(ROOT, "include"), os.path.join(root, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(root, "lib")
    path = tensors_path()
    tmp = path + ".tmp"
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + ["-I" + p for p in paths]
           + [os.path.join(CSRC, "tensors.cpp"), "-o", tmp, "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu",
              "-lc10"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for tensors.cpp:\n{r.stderr}")
    os.replace(tmp, path)


def _fresh(path: str) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()


def _build_library(verbose_ptxas: bool) -> None:
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc()] + ARCH + FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose_ptxas:
        for _, err in results:
            print(err)
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)

    def tensors():
        if force or not _fresh(tensors_path()):
            _build_tensors()

    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(tensors)
        if force or not _fresh(LIB):
            _build_library(verbose_ptxas)
        error = module.exception()
    if error is not None:
        warnings.warn(f"the paged and packed operators are not available: {error}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
