"""Build step for the CUDA library: compiles ``csrc/onebit_adam.cu`` for sm_100a into
``libonebit_adam.so`` next to this file (in-tree, so the built library travels with the repo), and
``csrc/binding.cpp``, the binding's native part for lists of tensors, into ``_binding.so``. The
library needs neither torch nor Python's headers; the binding's part is left out where they are
missing, and the functions that need it then raise.

Run ``python -m communication_compressed_optimizer_momentum_b200.build`` or call ``build()``.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC_DIR = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libonebit_adam.so")
SOURCES = [os.path.join(SRC_DIR, "onebit_adam.cu")]
DEPS = SOURCES + [os.path.join(SRC_DIR, "kernels.cuh"), os.path.join(SRC_DIR, "kernels_dp.cuh"),
                  os.path.join(SRC_DIR, "kernels_zero_one.cuh"),
                  os.path.join(SRC_DIR, "kernels_adamw.cuh"), os.path.join(SRC_DIR, "adamw.cuh"),
                  os.path.join(SRC_DIR, "adamw_clip.h"),
                  os.path.join(INCLUDE, "onebit_adam.h")]

# --fmad=false: no contraction of the method's fp32 multiply-adds (every fp32 operation is one
# IEEE operation); fp64 fused multiply-adds are written out where wanted. No fast-math, so
# division and square root are the correctly rounded ones.
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17", "--fmad=false",
    "-Xcompiler", "-fPIC", "-shared",
]


BINDING = os.path.join(PKG, "_binding.so")
BINDING_STAMP = BINDING + ".stamp"
BINDING_SOURCE = os.path.join(SRC_DIR, "binding.cpp")


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in DEPS)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library (and the binding's native part, where it can be) if it is missing or older
    than its sources; return the library's path."""
    if force or stale():
        build_library(verbose)
    if can_build_binding():
        build_binding(force)
    return LIB


def build_library(verbose: bool = False) -> None:
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", SRC_DIR, "-o", tmp, *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)


def can_build_binding() -> bool:
    """Whether torch and Python's headers are there."""
    import importlib.util
    import sysconfig
    return importlib.util.find_spec("torch") is not None and \
        os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))


def binding_command(out: str) -> list:
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    includes = [INCLUDE, os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(root, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()),
            *["-I" + p for p in includes], "-o", out, BINDING_SOURCE, "-L" + lib,
            "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def binding_stamp() -> str:
    """What the native part is good for: the Python, the torch and the command it was built with
    (wherever the tree lies: it may be moved)."""
    import torch
    command = " ".join(binding_command("_binding.so")).replace(ROOT + os.sep, "")
    return "\n".join([sys.implementation.cache_tag, torch.__version__, command]) + "\n"


def binding_stale() -> bool:
    """Missing, older than its sources, or of another Python, torch or command."""
    deps = (BINDING_SOURCE, os.path.join(SRC_DIR, "adamw_clip.h"),
            os.path.join(INCLUDE, "onebit_adam.h"))
    if not os.path.exists(BINDING) or \
            any(os.path.getmtime(p) > os.path.getmtime(BINDING) for p in deps):
        return True
    try:
        with open(BINDING_STAMP) as f:
            return f.read() != binding_stamp()
    except OSError:
        return True


def build_binding(force: bool = False) -> str:
    """Compile the binding's native part if it is stale."""
    if force or binding_stale():
        tmp = BINDING + ".tmp%d" % os.getpid()
        subprocess.check_call(binding_command(tmp))
        os.replace(tmp, BINDING)
        with open(BINDING_STAMP + ".tmp%d" % os.getpid(), "w") as f:
            f.write(binding_stamp())
        os.replace(f.name, BINDING_STAMP)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
