"""More of AdamW without a GPU: lengths beyond 64 bits, parameters that no step would take, a
host without memory, and what is built where."""
import os
import subprocess
import sys

import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("n", [1 << 63, (1 << 64) - 1, 1 << 64, (1 << 64) + 300, -(1 << 63) - 1,
                               -(1 << 64) + 5])
def test_layout_refuses_lengths_beyond_64_bits(n):
    with pytest.raises(ob.OneBitError, match="size"):
        ob.onebit_adamw_layout([5, n])


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32, torch.complex64])
@pytest.mark.parametrize("state", ["q8", "f32"])
def test_an_optimizer_refuses_parameters_that_its_step_would(dtype, state):
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ob.AdamW([torch.zeros(8, dtype=dtype)], state=state)
    with pytest.raises(TypeError, match="list of tensors"):
        ob.AdamW([1.0], state=state)


# 30 million empty tensors: their address ranges need 720 MB where 100 MB are left. Nothing is queued.
NO_MEMORY = r"""
import ctypes, resource, sys
sys.path.insert(0, %r)
import numpy as np
from communication_compressed_optimizer_momentum_b200 import _abi
L = _abi.lib()
n = 30_000_000
held = np.zeros(n, dtype=np.int64)
zeros = held.ctypes.data
assert L.onebit_grad_norm(1, zeros, zeros, 0, -1.0, 0, None, None) == -1
assert b"max_norm" in L.onebit_last_error()
size = [int(x.split()[1]) * 1024 for x in open("/proc/self/status") if x.startswith("VmSize")][0]
resource.setrlimit(resource.RLIMIT_AS, (size + 100_000_000, resource.RLIM_INFINITY))
rc = L.onebit_grad_norm(n, zeros, zeros, 0, 1.0, 0, 0x100000, None)
print(rc, L.onebit_last_error().decode())
""" % ROOT


def test_a_host_without_memory_gives_its_own_reason():
    """Not the reason of the call before; no exception leaves the C entry point."""
    r = subprocess.run([sys.executable, "-c", NO_MEMORY], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split(None, 1) == ["-5", "no host memory\n"], \
        r.stdout + r.stderr


# build.py by itself, as a program without torch or Python's headers uses it; the compilers' commands
# are recorded, not run.
BUILD = r"""
import importlib.util, subprocess, sys, sysconfig
missing, pkg = sys.argv[1], sys.argv[2]
spec = importlib.util.spec_from_file_location("build_alone", pkg + "/build.py")
build = importlib.util.module_from_spec(spec)
spec.loader.exec_module(build)
if missing == "torch":
    class NoTorch:
        def find_spec(self, name, path=None, target=None):
            if name.split(".")[0] == "torch":
                raise ModuleNotFoundError(name)
    sys.meta_path.insert(0, NoTorch())
    find = importlib.util.find_spec
    importlib.util.find_spec = lambda name, *a: None if name == "torch" else find(name, *a)
elif missing == "headers":
    paths = sysconfig.get_paths()
    sysconfig.get_paths = lambda *a, **k: dict(paths, include="/nonexistent")
ran = []
build.subprocess.check_call = lambda cmd, **k: ran.append(cmd[0].split("/")[-1])
build.os.replace = lambda a, b: ran.append("-> " + b.split("/")[-1])
assert build.build(force=True) == build.LIB
print(ran)
"""


@pytest.mark.parametrize("missing,want", [
    ("torch", ["nvcc", "-> libonebit_adam.so"]), ("headers", ["nvcc", "-> libonebit_adam.so"]),
    ("nothing", ["nvcc", "-> libonebit_adam.so", "g++", "-> _binding.so"])])
def test_the_library_is_built_without_torch(missing, want):
    pkg = os.path.join(ROOT, "communication_compressed_optimizer_momentum_b200")
    r = subprocess.run([sys.executable, "-c", BUILD, missing, pkg], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == repr(want), r.stdout + r.stderr
