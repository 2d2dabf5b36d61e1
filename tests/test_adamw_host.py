"""AdamW over a list of tensors without a GPU: the layout, every refusal of the C entry points
(which come before any device work) and of the binding, and the random bits of the 8-bit states'
stochastic rounding."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob
from adamw_reference import random_words
from communication_compressed_optimizer_momentum_b200 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from communication_compressed_optimizer_momentum_b200 import build
    build.build()
    return _abi.lib()


def test_layout():
    assert ob.onebit_adamw_layout([]) == ([], 0)
    assert ob.onebit_adamw_layout([0]) == ([0], 0)
    assert ob.onebit_adamw_layout([1, 0, 256, 257, 1 << 33]) == (
        [0, 256, 256, 512, 1024], 1024 + (1 << 33))
    with pytest.raises(ob.OneBitError, match="size"):
        ob.onebit_adamw_layout([-1])
    with pytest.raises(ob.OneBitError, match="size"):
        ob.onebit_adamw_layout([(1 << 39) + 1])


# Addresses are made up: every call below is refused on the host, before they are used. Each
# tensor has its own 64 KiB.
AT = {"p0": 0x10000, "p1": 0x20000, "g0": 0x30000, "g1": 0x40000, "c0": 0x50000, "c1": 0x60000,
      "m": 0x70000, "v": 0x90000, "ctl": 0xB0000, "scale": 0xC0000, "lr": 0xD0000,
      "me": 0xE0000, "ve": 0xF0000}


def pointers(*names_or_addresses):
    vals = [AT[x] if isinstance(x, str) else x for x in names_or_addresses]
    return (ctypes.c_void_p * len(vals))(*vals)


def call_step(lib, eight, **kw):
    a = dict(n=2, numel=[1000, 300], p=("p0", "p1"), ptype=0, g=("g0", "g1"), gtype=0, c=None,
             m=AT["m"], v=AT["v"], me=AT["me"], ve=AT["ve"], ctl=AT["ctl"], wd=[0.1, 0.0],
             scale=AT["scale"], lr_dev=AT["lr"], lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, bc=1)
    assert set(kw) <= set(a)
    a.update(kw)

    def arr(t, x):
        return None if x is None else (t * len(x))(*x)
    head = [a["n"], arr(ctypes.c_int64, a["numel"]), a["p"] and pointers(*a["p"]), a["ptype"],
            a["g"] and pointers(*a["g"]), a["gtype"], a["c"] and pointers(*a["c"])]
    tail = [arr(ctypes.c_double, a["wd"]), a["scale"], a["lr_dev"], a["lr"], a["b1"], a["b2"],
            a["eps"], a["bc"], None]
    if eight:
        rc = lib.onebit_adamw8_step(*head, a["m"], a["v"], a["me"], a["ve"], a["ctl"], 7, *tail)
    else:
        rc = lib.onebit_adamw_step(*head, a["m"], a["v"], a["ctl"], *tail)
    return rc, lib.onebit_last_error().decode()


nan, inf = float("nan"), float("inf")
REFUSED = [
    (dict(n=-1), -1, "negative"),
    (dict(numel=None), -1, "null list"),
    (dict(g=None), -1, "null list"),
    (dict(p=None), -1, "null list"),
    (dict(ptype=2), -1, "type"),
    (dict(gtype=-1), -1, "type"),
    (dict(numel=[-1, 3]), -1, "size"),
    (dict(numel=[3, (1 << 39) + 1]), -1, "size"),
    (dict(p=("p0", 0)), -1, "null tensor"),
    (dict(g=(0, "g1")), -1, "null tensor"),
    (dict(c=("c0", 0)), -1, "null tensor"),
    (dict(c=("c0", "c1"), ptype=1), -1, "float32"),
    (dict(p=(0x10002, "p1")), -2, "aligned"),
    (dict(g=("g0", 0x40001), gtype=1), -2, "aligned"),
    (dict(c=("c0", 0x60001)), -2, "aligned"),
    (dict(m=AT["m"] + 4), -2, "aligned"),
    (dict(v=AT["v"] + 8), -2, "aligned"),
    (dict(ctl=AT["ctl"] + 4), -2, "aligned"),
    (dict(scale=AT["scale"] + 2), -2, "aligned"),
    (dict(lr_dev=AT["lr"] + 4), -2, "aligned"),
    (dict(m=None), -1, "null state"),
    (dict(v=None), -1, "null state"),
    (dict(ctl=None), -1, "null ctl"),
    (dict(wd=[0.1, -0.1]), -1, "decay"),
    (dict(wd=[nan, 0.1]), -1, "decay"),
    (dict(wd=[inf, 0.1]), -1, "decay"),
    (dict(lr=inf), -1, "lr"),
    (dict(lr=nan), -1, "lr"),
    (dict(b1=1.0), -1, "beta"),
    (dict(b2=-0.1), -1, "beta"),
    (dict(b2=nan), -1, "beta"),
    (dict(eps=-1e-8), -1, "eps"),
    (dict(eps=inf), -1, "eps"),
    (dict(bc=2), -1, "bias"),
    (dict(p=("p0", "p0")), -1, "overlap"),                    # the same parameter twice
    (dict(p=("p0", AT["p0"] + 3996)), -1, "overlap"),         # by one element
    (dict(g=("g0", "p0")), -1, "overlap"),                    # a gradient in a parameter
    (dict(g=("p0", "g1")), -1, "overlap"),
    (dict(c=("c0", "g1")), -1, "overlap"),
    (dict(c=("c0", "c0")), -1, "overlap"),
    (dict(m=AT["v"]), -1, "overlap"),
    (dict(v=AT["m"] + 1024), -1, "overlap"),
    (dict(p=("p0", AT["m"] + 32)), -1, "overlap"),
    (dict(ctl=AT["p1"] + 8), -1, "overlap"),
    (dict(scale=AT["ctl"] + 40), -1, "overlap"),
    (dict(lr_dev=AT["p0"]), -1, "overlap"),
]


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "q8"])
@pytest.mark.parametrize("change,code,why", REFUSED, ids=[str(k) for k in range(len(REFUSED))])
def test_step_refusals(lib, eight, change, code, why):
    rc, text = call_step(lib, eight, **change)
    assert (rc, why in text) == (code, True), (rc, text)


def test_states_alignment(lib):
    """fp32 states are read 32 bytes at a time, exponents four at a time, codes 16-byte aligned."""
    assert call_step(lib, False, m=AT["m"] + 16)[0] == -2
    assert call_step(lib, False, v=AT["v"] + 16)[0] == -2
    assert call_step(lib, True, me=AT["me"] + 2)[0] == -2
    assert call_step(lib, True, ve=AT["ve"] + 1)[0] == -2


def test_step8_refuses_missing_or_overlapping_exponents(lib):
    assert call_step(lib, True, me=None)[0] == -1
    assert call_step(lib, True, ve=None)[0] == -1
    rc, text = call_step(lib, True, ve=AT["me"] + 4)          # 4 + 2 blocks: 6 exponents
    assert rc == -1 and "overlap" in text
    rc, text = call_step(lib, True, me=AT["m"])
    assert rc == -1 and "overlap" in text


def call_norm(lib, n=2, numel=(1000, 300), g=("g0", "g1"), gtype=0, max_norm=1.0, acc=0,
              work=0x100000):
    rc = lib.onebit_grad_norm(n, (ctypes.c_int64 * len(numel))(*numel) if numel else None,
                              g and pointers(*g), gtype, max_norm, acc, work, None)
    return rc, lib.onebit_last_error().decode()


@pytest.mark.parametrize("change,code,why", [
    (dict(n=-1), -1, "negative"), (dict(numel=None), -1, "null list"),
    (dict(g=None), -1, "null list"), (dict(gtype=5), -1, "type"),
    (dict(max_norm=0.0), -1, "max_norm"), (dict(max_norm=-1.0), -1, "max_norm"),
    (dict(max_norm=nan), -1, "max_norm"), (dict(acc=2), -1, "accumulate"),
    (dict(work=None), -1, "null work"), (dict(work=0x100004), -2, "aligned"),
    (dict(g=("g0", 0)), -1, "null tensor"), (dict(g=("g0", 0x40002)), -2, "aligned"),
    (dict(work=AT["g1"] - 16384 + 8), -1, "overlap"),
], ids=lambda x: None)
def test_norm_refusals(lib, change, code, why):
    rc, text = call_norm(lib, **change)
    assert (rc, why in text) == (code, True), (rc, text)


@pytest.mark.parametrize("which", ["get", "set"])
@pytest.mark.parametrize("change,code", [
    (dict(total=-256), -1), (dict(total=100), -1), (dict(a=None, b=None), -1),
    (dict(mc=None), -1), (dict(vk=None), -1), (dict(mc=0x1008), -2), (dict(a=0x50008), -2),
    (dict(b=0x60010), -2), (dict(mk=0x3002), -2),
    (dict(b=0x50100), -1),                                    # the two values overlap
    (dict(a=0x1100), -1),                                     # a value in the codes
], ids=lambda x: None)
def test_state8_refusals(lib, which, change, code):
    a = dict(total=1024, mc=0x1000, vc=0x2000, mk=0x3000, vk=0x4000, a=0x50000, b=0x60000)
    a.update(change)
    if which == "set" and change == dict(b=0x50100):
        pytest.skip("sources may share memory")
    args = [a["total"], a["mc"], a["vc"], a["mk"], a["vk"], a["a"], a["b"]]
    rc = lib.onebit_adamw8_get_state(*args, 0, None) if which == "get" else \
        lib.onebit_adamw8_set_state(*args, None)
    assert rc == code


def test_state8_empty_and_type(lib):
    assert lib.onebit_adamw8_get_state(0, None, None, None, None, None, None, 0, None) == 0
    assert lib.onebit_adamw8_set_state(0, None, None, None, None, None, None, None) == 0
    assert lib.onebit_adamw8_get_state(256, 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 2,
                                       None) == -1


def test_binding_refuses_host_tensors_and_wrong_kinds():
    x = torch.zeros(8)
    ctl = torch.zeros(8, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        ob.onebit_adamw_step([x], [x], x, x, ctl, 1e-3)
    with pytest.raises(ValueError, match="1 gradients for 2"):
        ob.onebit_adamw_step([x, x], [x], x, x, ctl, 1e-3)
    with pytest.raises(ValueError, match="CUDA"):
        ob.onebit_grad_norm([x])
    with pytest.raises(ValueError, match="no gradients"):
        ob.onebit_grad_norm([])
    with pytest.raises(ValueError, match="accumulate"):
        ob.onebit_grad_norm([x], accumulate=True)
    with pytest.raises(TypeError, match="list of tensors"):
        ob.onebit_grad_norm([1.0])
    with pytest.raises(ValueError, match="CUDA"):
        ob.onebit_adamw8_get_state(*[x.to(torch.uint8)] * 4)
    with pytest.raises(ValueError, match="CUDA"):
        ob.AdamW([x])
    with pytest.raises(ValueError, match="no parameters"):
        ob.AdamW([])
    with pytest.raises(ValueError, match="f32"):
        ob.AdamW([x], state="f16")


MISSING = r'''
import sys
sys.path.insert(0, %r)
import torch
from communication_compressed_optimizer_momentum_b200 import _abi
_abi.LIB_PATH = "/nonexistent/libonebit_adam.so"
import communication_compressed_optimizer_momentum_b200 as ob
x, q = torch.zeros(256), torch.zeros(256, dtype=torch.uint8)
for name, fn in {
        "layout": lambda: ob.onebit_adamw_layout([3]),
        "step": lambda: ob.onebit_adamw_step([x], [x], x, x, x, 1e-3),
        "step8": lambda: ob.onebit_adamw8_step([x], [x], q, q, q, q, x, 1e-3),
        "get": lambda: ob.onebit_adamw8_get_state(q, q, q, q),
        "set": lambda: ob.onebit_adamw8_set_state(q, q, q, q, x, x),
        "norm": lambda: ob.onebit_grad_norm([x])}.items():
    try:
        fn()
    except RuntimeError as e:
        assert "not built" in str(e), (name, str(e))
        continue
    raise SystemExit("%%s did not raise" %% name)
print("all raised")
''' % ROOT


def test_every_function_raises_without_the_library():
    r = subprocess.run([sys.executable, "-c", MISSING], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all raised" in r.stdout, r.stdout + r.stderr


# ----------------------------------------------------------------------------------------------
# The documented random bits (the GPU tests compare the kernels' roundings with the same formula)

def test_random_bits_are_uniform_and_uncorrelated():
    """Means, bits and correlations of the 16-bit numbers over places, steps and seeds stay within
    5 standard errors of those of independent uniform ones (about 100 comparisons: a correct
    generator fails one with probability 6e-5; the input is fixed)."""
    n = 1 << 18
    base = random_words(np.arange(n), 3, 1)
    streams = {"place": base, "next step": random_words(np.arange(n), 3, 2),
               "next seed": random_words(np.arange(n), 4, 1),
               "far": random_words(np.arange(n) + (1 << 36), 3, 1)}

    def halves(x):
        return [(x >> 16).astype(np.float64) / 65536, (x & 0xFFFF).astype(np.float64) / 65536]
    cols = [(name + h, v) for name, x in streams.items() for h, v in zip("mv", halves(x))]
    sd = math.sqrt(1 / 12)
    for name, v in cols:
        assert abs(v.mean() - (0.5 - 2 ** -17)) < 5 * sd / math.sqrt(n), name
        for lag in (1, 7, 8, 256):
            c = np.mean((v[lag:] - 0.5) * (v[:-lag] - 0.5)) * 12
            assert abs(c) < 5 / math.sqrt(n), (name, lag, c)
    for a in range(len(cols)):
        for b in range(a):
            c = np.mean((cols[a][1] - 0.5) * (cols[b][1] - 0.5)) * 12
            assert abs(c) < 5 / math.sqrt(n), (cols[a][0], cols[b][0], c)
    bits = ((base[:, None] >> np.arange(32, dtype=np.uint32)) & 1).mean(0)
    assert np.abs(bits - 0.5).max() < 5 * 0.5 / math.sqrt(n)
