"""Build the in-tree CUDA library ``libw4a16.so`` for sm_100a with nvcc, and the native part of
the Python binding, ``w8_native.<key>.so``, with the host compiler."""
from __future__ import annotations

import glob
import hashlib
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libw4a16.so")
INCLUDE = os.path.join(ROOT, "include")
BINDING = os.path.join(HERE, "binding", "w8_native.cpp")
BINDING_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden"]
BINDING_LIBS = ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, f"-I{INCLUDE}", os.path.join(CSRC, "w4a16.cu"), "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def _binding_abi() -> str:
    import torch
    return f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def binding_path() -> str:
    """Where the binding for this interpreter, this PyTorch and these sources lies.  The module uses
    PyTorch's C++ internals, so a file that was built against another must not be loaded."""
    import sysconfig

    import torch
    key = hashlib.sha256()
    for part in (sysconfig.get_config_var("SOABI"), torch.__version__, torch.version.cuda, _binding_abi(),
                 *BINDING_FLAGS, *BINDING_LIBS):
        key.update(f"{part}\0".encode())
    for source in (BINDING, os.path.join(INCLUDE, "w4a16.h")):
        with open(source, "rb") as f:
            key.update(hashlib.sha256(f.read()).digest())
    return os.path.join(HERE, f"w8_native.{key.hexdigest()[:12]}.so")


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The native calls of the binding: a CPython module against PyTorch's headers.  It reaches
    the CUDA library through function addresses, so it does not link to it."""
    path = binding_path()
    if not force and os.path.exists(path):
        return path
    import sysconfig

    from torch.utils import cpp_extension
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    includes = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths(), cuda]
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), *BINDING_FLAGS, _binding_abi(), *[f"-I{d}" for d in includes], BINDING,
           "-o", tmp, *[f"-L{d}" for d in cpp_extension.library_paths()], *BINDING_LIBS]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, path)
    return path


if __name__ == "__main__":
    print(build_binding(force="--force" in sys.argv, verbose=True))
    print(build(force="--force" in sys.argv, verbose=True))
