"""Build the StreamKL CUDA library in-tree for sm_100a.

    python -m attention_kl_divergence_fwd_b200.build [--verbose]

Compiles csrc/streamkl_api.cu (which includes every kernel) with nvcc into
``attention_kl_divergence_fwd_b200/lib/libstreamkl.so``. The CUDA runtime is linked
statically and the driver API is reached through the runtime's entry-point query,
so the library loads on hosts without a GPU driver (only launching needs a GPU).

csrc/sparse_dispatch.cpp, the PyTorch side of the block-sparse calls, becomes
``lib/_sparse_dispatch.so``; it reaches the library through addresses handed over at run time.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIB_DIR, "libstreamkl.so")
SOURCES = [os.path.join(PKG, "csrc", "streamkl_api.cu")]
DISPATCH = os.path.join(LIB_DIR, "_sparse_dispatch.so")
DISPATCH_SOURCE = os.path.join(PKG, "csrc", "sparse_dispatch.cpp")
DEPS = [os.path.join(PKG, "csrc", f) for f in os.listdir(os.path.join(PKG, "csrc"))
        if not f.endswith(".cpp")] + [os.path.join(ROOT, "include", "streamkl.h")]

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in DEPS if os.path.exists(p))


def build_dispatch(force: bool = False, verbose: bool = False) -> str:
    from .sparse import dispatch_current
    deps = [DISPATCH_SOURCE, os.path.join(ROOT, "include", "streamkl.h")]
    stale = not dispatch_current() or any(
        os.path.getmtime(p) > os.path.getmtime(DISPATCH) for p in deps)
    if not force and not stale:
        return DISPATCH
    try:
        _compile_dispatch(verbose)
    except (OSError, RuntimeError):
        if stale and os.path.exists(DISPATCH):  # of other sources or another PyTorch: better none
            os.remove(DISPATCH)
        raise
    return DISPATCH


def _compile_dispatch(verbose: bool) -> None:
    import torch
    from .sparse import dispatch_marker
    base = os.path.dirname(torch.__file__)
    include = [os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
               os.path.join(ROOT, "include")]
    lib = os.path.join(base, "lib")
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = DISPATCH + ".tmp"
    # The compiler that nvcc uses: one that links libstdc++ statically would put a second copy
    # beside PyTorch's, and the two break each other's streams.
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DBUILT_FOR="{dispatch_marker()}"', "-DTORCH_EXTENSION_NAME=_sparse_dispatch",
           "-DTORCH_API_INCLUDE_EXTENSION_H",
           *(f"-I{p}" for p in include), DISPATCH_SOURCE, "-o", tmp, f"-L{lib}", "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{cmd[0]} failed with exit code {res.returncode}")
    os.replace(tmp, DISPATCH)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, and the dispatch module where it can be built: without g++, Python's headers or
    a CUDA build of PyTorch the block-sparse calls raise OSError and everything else works."""
    if force or not up_to_date():
        _compile_library(verbose)
    try:
        build_dispatch(force, verbose)
    except (OSError, RuntimeError) as e:
        warnings.warn(f"the block-sparse calls are not available: {e}")
    return LIB


def _compile_library(verbose: bool) -> None:
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I",
           os.path.join(PKG, "csrc"), *SOURCES, "-o", tmp]
    if verbose:
        cmd += ["-Xptxas", "-v"]
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed with exit code {res.returncode}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
