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
import importlib.util, os, subprocess, sys, sysconfig
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
def replace(a, b):
    if os.path.exists(a):                             # the note of what it was built with
        os.remove(a)
    else:
        ran.append("-> " + b.split("/")[-1])
build.os.replace = replace
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


def test_the_native_part_is_stale_with_another_torch_python_or_command(tmp_path, monkeypatch):
    from communication_compressed_optimizer_momentum_b200 import build
    build.build()
    assert not build.binding_stale()                  # as it was built
    built = tmp_path / "_binding.so"
    built.write_bytes(b"")
    monkeypatch.setattr(build, "BINDING", str(built))
    monkeypatch.setattr(build, "BINDING_STAMP", str(built) + ".stamp")
    assert build.binding_stale()                      # nothing says what it was built with
    commands = []
    monkeypatch.setattr(build.subprocess, "check_call", lambda cmd: commands.append(cmd) or open(
        cmd[cmd.index("-o") + 1], "w").close())
    build.build_binding()
    assert len(commands) == 1 and not build.binding_stale()
    build.build_binding()
    assert len(commands) == 1                         # nothing to do
    with monkeypatch.context() as other:
        other.setattr(torch, "__version__", "9.9")
        assert build.binding_stale()
    with monkeypatch.context() as other:
        other.setattr(build, "nvcc", lambda: "/opt/other/cuda/bin/nvcc")
        assert build.binding_stale()
    assert not build.binding_stale()
    with monkeypatch.context() as moved:              # the whole tree at another place
        for name in ("ROOT", "PKG", "SRC_DIR", "INCLUDE", "BINDING_SOURCE"):
            moved.setattr(build, name, getattr(build, name).replace(ROOT, "/else/where"))
        stamp = build.binding_stamp()
    assert stamp == build.binding_stamp() and ROOT not in stamp
    monkeypatch.setattr(build.sys, "implementation", type("Other", (), {"cache_tag": "cpython-399"}))
    assert build.binding_stale()
    build.build_binding()
    assert len(commands) == 2 and not build.binding_stale()


UNLOADABLE = r"""
import sys
sys.path.insert(0, sys.argv[1])
import communication_compressed_optimizer_momentum_b200 as ob
import torch
try:
    ob.onebit_grad_norm([torch.zeros(3)])
except RuntimeError as e:
    print(e)
"""


@pytest.mark.parametrize("content,want", [(None, "not built"), (b"of another torch", "cannot be loaded")])
def test_a_native_part_that_does_not_load_is_told_from_a_missing_one(tmp_path, content, want):
    """In a copy of the package, whose _binding.so is missing or no library at all."""
    name = "communication_compressed_optimizer_momentum_b200"
    pkg = tmp_path / name
    pkg.mkdir()
    for f in os.listdir(os.path.join(ROOT, name)):
        if f.endswith(".py") or f == "libonebit_adam.so":
            os.symlink(os.path.join(ROOT, name, f), pkg / f)
    if content is not None:
        (pkg / "_binding.so").write_bytes(content)
    r = subprocess.run([sys.executable, "-c", UNLOADABLE, str(tmp_path)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "_binding.so " in r.stdout and want in r.stdout, r.stdout + r.stderr
