"""Builds, in-tree, libpbsa.so (the C ABI of include/pbsa.h) for sm_100a with nvcc and
token_calls.so (a CPython module over torch's tensors) with the host compiler."""
from __future__ import annotations

import glob
import os
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libpbsa.so")
CALLS = os.path.join(PKG, "token_calls.so")
CALLS_SOURCE = os.path.join(PKG, "csrc", "token_calls.cpp")
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-shared", "--threads", "0", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cuh")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def library_up_to_date() -> bool:
    return os.path.exists(LIB) and all(os.path.getmtime(f) <= os.path.getmtime(LIB) for f in sources() + headers())


def calls_up_to_date() -> bool:
    """Whether the module is newer than its sources and reads this torch's tensors."""
    import torch
    if not os.path.exists(CALLS) or any(os.path.getmtime(f) > os.path.getmtime(CALLS)
                                        for f in headers() + [CALLS_SOURCE]):
        return False
    with open(CALLS, "rb") as f:
        return f"token_calls for torch {torch.__version__}\0".encode() in f.read()


def up_to_date() -> bool:
    return library_up_to_date() and calls_up_to_date()


def calls_command():
    import torch
    from torch.utils import cpp_extension
    includes = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            f'-DTORCH_VERSION_BUILT="{torch.__version__}"',
            "-I", os.path.join(ROOT, "include"), *(x for d in includes for x in ("-isystem", d)),
            "-o", CALLS + ".tmp", CALLS_SOURCE, "-L", PKG, "-lpbsa",
            *(x for d in cpp_extension.library_paths() for x in ("-L", d)),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]


def build_calls(verbose: bool = False) -> bool:
    """Compiles the module beside the library.  Where that fails (no headers of torch or Python)
    none is left, and pbsa.py makes every call through ctypes."""
    try:
        cmd = calls_command()
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        os.replace(CALLS + ".tmp", CALLS)
        return True
    except (OSError, ImportError, subprocess.CalledProcessError) as e:
        if os.path.exists(CALLS):
            os.remove(CALLS)
        warnings.warn(f"token_calls.so could not be built ({e})")
        return False


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ into one shared library, and the module beside it; returns
    the library's path."""
    if force or not library_up_to_date():
        nvcc = os.environ.get("NVCC", "nvcc")
        cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-o", LIB + ".tmp", *sources()]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        os.replace(LIB + ".tmp", LIB)
    if force or not calls_up_to_date():
        build_calls(verbose)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
