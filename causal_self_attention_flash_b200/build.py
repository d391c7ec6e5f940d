"""Build libcattn.so (sm_100a) in-tree with nvcc, and _torch_calls-*.so, the
Python binding's argument marshalling, with the host compiler.

    python causal_self_attention_flash_b200/build.py [--force]

Both land next to this file, so they travel with the source tree.  The second
holds for one Python and one torch, which its name tells; the package does
without it, at some microseconds a call.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libcattn.so")

SOURCES = ["api.cu"]
BINDING_SOURCE = "torch_calls.cpp"
# every device source and header: a change to any of them rebuilds
DEPS = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared", "-cudart", "shared",
]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    files = [os.path.join(CSRC, f) for f in DEPS] + [os.path.join(INCLUDE, "cattn.h"),
                                                    os.path.abspath(__file__)]
    return any(os.path.getmtime(f) > t for f in files)


def binding_path() -> str:
    """Where the binding for this Python and the installed torch is (_binding.py
    looks for the same name)."""
    import torch
    return os.path.join(
        HERE, f"_torch_calls-{sys.implementation.cache_tag}-torch{torch.__version__}.so")


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The binding, against the headers of the installed torch."""
    src, out = os.path.join(CSRC, BINDING_SOURCE), binding_path()
    files = [src, os.path.abspath(__file__)]
    if not force and os.path.exists(out) and \
            all(os.path.getmtime(f) <= os.path.getmtime(out) for f in files):
        return out
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    lib = os.path.join(root, "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(cuda, "include"), src, "-L", lib, f"-Wl,-rpath,{lib}",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-o", out + ".tmp"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(out + ".tmp", out)
    return out


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _stale():
        cmd = [nvcc_path(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC,
               *[os.path.join(CSRC, s) for s in SOURCES], "-o", LIB + ".tmp"]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        os.replace(LIB + ".tmp", LIB)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
