"""Builds libdsa.so (the CUDA kernels and their C-ABI) in-tree for sm_100a with nvcc and, where torch
is installed, _calls.so (native argument marshalling for the Python binding) beside it with g++.

    python -m sparse_long_context_dsa_b200.build [--force]
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdsa.so")
CALLS = os.path.join(HERE, "_calls.so")
CALLS_TORCH = os.path.join(HERE, "_build", "calls_torch.txt")      # the torch version that _calls.so was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-shared", "-Xptxas", "-warn-spills"]


def sources():
    out = [os.path.join(ROOT, "include", "dsa.h")]
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh")):
            out.append(os.path.join(CSRC, f))
    return out


def torch_version():
    """The installed torch's version, None without one (its headers' ABI is the extension's)."""
    from importlib import metadata
    try:
        return metadata.version("torch")
    except metadata.PackageNotFoundError:
        pass
    try:                               # a torch without package metadata
        import torch
        return str(torch.__version__)
    except ImportError:
        return None


def calls_stale() -> bool:
    """Whether _calls.so is older than its sources or was built for another torch."""
    src = [os.path.join(CSRC, "calls.cpp"), os.path.join(ROOT, "include", "dsa.h")]
    if not os.path.exists(CALLS) or os.path.getmtime(CALLS) < max(os.path.getmtime(s) for s in src):
        return True
    try:
        with open(CALLS_TORCH) as f:
            return f.read().strip() != torch_version()
    except FileNotFoundError:
        return True


def build_calls(force: bool = False, verbose: bool = False) -> str:
    if not force and not calls_stale():
        return CALLS
    import sysconfig
    import torch
    t = os.path.dirname(torch.__file__)
    tmp = CALLS + f".tmp{os.getpid()}"
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", *["-I" + i for i in inc],
           os.path.join(CSRC, "calls.cpp"), "-o", tmp,
           "-L" + os.path.join(t, "lib"), "-Wl,-rpath," + os.path.join(t, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, CALLS)
    os.makedirs(os.path.dirname(CALLS_TORCH), exist_ok=True)
    with open(CALLS_TORCH, "w") as f:
        f.write(torch_version() or "")
    return CALLS


def build_lib(force: bool = False, verbose: bool = False) -> str:
    """libdsa.so alone: nvcc and the sources are all it needs."""
    newest = max(os.path.getmtime(s) for s in sources())
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *FLAGS, "-o", tmp, os.path.join(CSRC, "dsa.cu")]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """libdsa.so and, where torch is installed (the Python binding needs it), _calls.so."""
    build_lib(force, verbose)
    if torch_version() is not None:
        build_calls(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
