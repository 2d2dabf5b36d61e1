"""Matrices in microscaled 4-bit floating point without a GPU: the layout, every refusal of the C
entry points (which come before any device work) and of the binding, and the reference itself."""
import ctypes

import numpy as np
import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob
import mx4_reference as ref
from communication_compressed_optimizer_momentum_b200 import _abi

ARG, ALIGN = -1, -2


@pytest.fixture(scope="module")
def lib():
    from communication_compressed_optimizer_momentum_b200 import build
    build.build()
    return _abi.lib()


def test_layout():
    assert ob.onebit_mx4_layout(0, 5) == (0, 0)
    assert ob.onebit_mx4_layout(5, 0) == (0, 0)
    assert ob.onebit_mx4_layout(1, 1) == (16, 512)
    assert ob.onebit_mx4_layout(128, 128) == (128 * 64, 512)
    assert ob.onebit_mx4_layout(129, 129) == (129 * 80, 4 * 512)
    assert ob.onebit_mx4_layout(1 << 30, 1 << 30) == (1 << 59, 1 << 55)
    for size in ((-1, 3), (3, -1), ((1 << 30) + 1, 3), (3, 1 << 40), (1 << 70, 3)):
        with pytest.raises(ob.OneBitError, match="size"):
            ob.onebit_mx4_layout(*size)


# Addresses are made up: every call below is refused on the host, before they are used. Each buffer
# has its own mebibyte.
AT = {n: (i + 1) << 20 for i, n in enumerate(
    ("x", "c", "s", "ct", "st", "e", "a", "as", "b", "bs", "out"))}


def quantize(lib, **kw):
    a = dict(rows=100, cols=70, x=AT["x"], dtype=0, ld=70, c=AT["c"], s=AT["s"], ct=AT["ct"],
             st=AT["st"], sr=0, seed=1, e=None, lde=70)
    assert set(kw) <= set(a)
    a.update(kw)
    rc = lib.onebit_mx4_quantize(*a.values(), None)
    return rc, lib.onebit_last_error().decode()


@pytest.mark.parametrize("kw,code,why", [
    (dict(rows=-1), ARG, "size"),
    (dict(cols=(1 << 30) + 1), ARG, "size"),
    (dict(rows=1 << 30, cols=1 << 30, ld=1 << 30, c=1 << 40, s=1 << 61, ct=None), ARG, "size"),
    (dict(dtype=2), ARG, "type"),
    (dict(sr=2), ARG, "stochastic"),
    (dict(x=None), ARG, "null x"),
    (dict(x=AT["x"] + 2), ALIGN, "x not aligned"),
    (dict(x=AT["x"] + 1, dtype=1), ALIGN, "x not aligned"),
    (dict(ld=69), ARG, "stride of x"),
    (dict(ld=0), ARG, "stride of x"),
    (dict(ld=-70), ARG, "stride of x"),
    (dict(c=None, ct=None), ARG, "neither"),
    (dict(s=None), ARG, "null codes"),
    (dict(st=None), ARG, "null codes"),
    (dict(c=AT["c"] + 8), ALIGN, "16-byte"),
    (dict(st=AT["st"] + 4), ALIGN, "16-byte"),
    (dict(e=AT["e"]), ARG, "residual goes"),
    (dict(e=AT["e"], c=None), ARG, "residual goes"),
    (dict(e=AT["e"], ct=None, lde=69), ARG, "stride of residual"),
    (dict(e=AT["e"] + 2, ct=None), ALIGN, "residual not aligned"),
    (dict(e=AT["x"], ct=None), ARG, "overlaps"),
    (dict(c=AT["x"]), ARG, "overlaps"),
    (dict(c=AT["x"] + 99 * 280 + 264), ARG, "overlaps"),
    (dict(s=AT["c"]), ARG, "overlaps"),
    (dict(ct=AT["c"]), ARG, "overlaps"),
    (dict(st=AT["s"]), ARG, "overlaps"),
])
def test_quantize_refuses(lib, kw, code, why):
    rc, text = quantize(lib, **kw)
    assert rc == code and why in text, (rc, text)


def test_empty_matrices_need_no_buffers(lib):
    for kw in (dict(rows=0), dict(cols=0)):
        assert quantize(lib, x=None, c=None, s=None, ct=None, st=None, **kw)[0] == 0
    assert lib.onebit_mx4_dequantize(0, 5, None, None, None, 0, 0, None) == 0
    assert lib.onebit_mx4_dequantize(5, 0, None, None, None, 1, 0, None) == 0
    assert lib.onebit_mx4_matmul(0, 5, 64, None, None, None, None, None, 0, 0, 0, None) == 0
    assert lib.onebit_mx4_matmul(5, 0, 64, None, None, None, None, None, 0, 0, 0, None) == 0
    assert lib.onebit_mx4_matmul(5, 3, 0, None, None, None, None, AT["out"], 0, 3, 1, None) == 0


def dequantize(lib, **kw):
    a = dict(rows=100, cols=70, c=AT["c"], s=AT["s"], out=AT["out"], dtype=0, ld=70)
    a.update(kw)
    rc = lib.onebit_mx4_dequantize(*a.values(), None)
    return rc, lib.onebit_last_error().decode()


@pytest.mark.parametrize("kw,code,why", [
    (dict(rows=-3), ARG, "size"),
    (dict(dtype=-1), ARG, "type"),
    (dict(c=None), ARG, "null codes"),
    (dict(s=AT["s"] + 1), ALIGN, "16-byte"),
    (dict(out=None), ARG, "null out"),
    (dict(out=AT["out"] + 1, dtype=1), ALIGN, "out not aligned"),
    (dict(ld=60), ARG, "stride of out"),
    (dict(out=AT["c"]), ARG, "overlaps"),
    (dict(out=AT["s"] - 4), ARG, "overlaps"),
])
def test_dequantize_refuses(lib, kw, code, why):
    rc, text = dequantize(lib, **kw)
    assert rc == code and why in text, (rc, text)


def matmul(lib, **kw):
    a = dict(m=100, n=200, k=70, a=AT["a"], sa=AT["as"], b=AT["b"], sb=AT["bs"], out=AT["out"],
             dtype=0, ld=200, acc=0)
    a.update(kw)
    rc = lib.onebit_mx4_matmul(*a.values(), None)
    return rc, lib.onebit_last_error().decode()


@pytest.mark.parametrize("kw,code,why", [
    (dict(m=-1), ARG, "size"),
    (dict(n=(1 << 30) + 1), ARG, "size"),
    (dict(k=-1), ARG, "size"),
    (dict(dtype=3), ARG, "type"),
    (dict(acc=2), ARG, "accumulate"),
    (dict(acc=1, dtype=1), ARG, "float32 out"),
    (dict(a=None), ARG, "null codes"),
    (dict(sb=None), ARG, "null codes"),
    (dict(sa=AT["as"] + 8), ALIGN, "16-byte"),
    (dict(b=AT["b"] + 1), ALIGN, "16-byte"),
    (dict(out=None), ARG, "null out"),
    (dict(out=None, k=0), ARG, "null out"),
    (dict(out=AT["out"] + 2), ALIGN, "out not aligned"),
    (dict(ld=199), ARG, "stride of out"),
    (dict(out=AT["a"]), ARG, "overlaps"),
    (dict(out=AT["bs"] - 8), ARG, "overlaps"),
])
def test_matmul_refuses(lib, kw, code, why):
    rc, text = matmul(lib, **kw)
    assert rc == code and why in text, (rc, text)


def test_status_refuses(lib):
    assert lib.onebit_mx4_status(None, None) == ARG
    assert "null" in lib.onebit_last_error().decode()


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ob.onebit_mx4_quantize(x)
    with pytest.raises(TypeError, match="Tensor"):
        ob.onebit_mx4_quantize([[0.0]])
    q = ob.Mx4.empty(4, 32, device="cpu")
    assert q.shape == (4, 32) and q.codes.numel() == 64 and q.scales.numel() == 512
    with pytest.raises(ValueError, match="CUDA tensor"):
        ob.onebit_mx4_dequantize(q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ob.onebit_mx4_matmul(q, q)
    with pytest.raises(TypeError, match="Mx4"):
        ob.onebit_mx4_matmul(x, q)
    with pytest.raises(TypeError, match="Mx4"):
        ob.onebit_mx4_quantize(x, out=x)
    with pytest.raises(ValueError, match="forms"):
        ob.onebit_mx4_quantize(x, forms="row")
    with pytest.raises(ValueError, match="rounding"):
        ob.onebit_mx4_quantize(x, rounding="up")
    with pytest.raises(ValueError, match="residual"):
        ob.onebit_mx4_quantize(x, forms="both", residual=x)
    with pytest.raises(TypeError, match="matrix"):
        ob.Mx4Linear(torch.zeros(5))
    with pytest.raises(ValueError, match="CUDA tensor"):
        ob.Mx4Linear(torch.zeros(5, 5))


def test_reference_by_hand():
    x = np.zeros((1, 40), dtype=np.float32)
    x[0, :8] = [6, -6, 5, 3.5, 2.5, 1.75, 0.25, -0.75]     # ties go to the even code
    x[0, 32:35] = [6.1, 12, 1]                             # 2^1
    code, e = ref.quantize(x)
    assert list(code[0, :8]) == [7, 15, 6, 6, 4, 4, 0, 10]
    assert e.tolist() == [[127, 128]]
    assert ref.values(code, e, 40)[0, 32:35].tolist() == [6, 12, 1]
    packed, scales = ref.pack(code, e)
    assert packed.shape == (1, 32) and packed[0, 0] == 7 | 15 << 4
    assert scales[:4].tolist() == [127, 128, 0, 0] and scales.size == 512


def test_random_bits_are_uniform_and_unrelated():
    """Means and correlations of a million of them: within five standard deviations."""
    n = 1 << 20
    u = [ref.random16(np.arange(n), s).astype(float) / 65536 - 0.5 for s in (0, 1, 2, 1 << 40)]
    sd = (1 / 12) ** 0.5
    for x in u:
        assert abs(x.mean()) < 5 * sd / n ** 0.5 + 2 ** -17
        for lag in (1, 2, 8, 32):
            assert abs((x[lag:] * x[:-lag]).mean()) < 5 * sd ** 2 / n ** 0.5
    for i in range(4):
        for j in range(i):
            assert abs((u[i] * u[j]).mean()) < 5 * sd ** 2 / n ** 0.5


def linear(lib, **kw):
    a = dict(m=100, n=200, k=70, x=AT["x"], xt=0, ldx=70, b=AT["b"], sb=AT["bs"], a=AT["a"], sa=AT["as"],
             at=AT["ct"], sat=AT["st"], out=AT["out"], dtype=1, ld=200)
    assert set(kw) <= set(a)
    a.update(kw)
    rc = lib.onebit_mx4_linear(*a.values(), None)
    return rc, lib.onebit_last_error().decode()


@pytest.mark.parametrize("kw,code,why", [
    (dict(m=-1), ARG, "size"),
    (dict(k=1 << 31), ARG, "size"),
    (dict(xt=3), ARG, "type"),
    (dict(dtype=-1), ARG, "type"),
    (dict(x=None), ARG, "null x"),
    (dict(x=AT["x"] + 2), ALIGN, "x not aligned"),
    (dict(ldx=69), ARG, "stride of x"),
    (dict(b=None), ARG, "null codes"),
    (dict(sb=AT["bs"] + 4), ALIGN, "16-byte"),
    (dict(a=None), ARG, "null codes"),
    (dict(a=None, at=None), ARG, "null codes"),
    (dict(m=4, a=None), ARG, "null codes"),             # with the transposed form, memory is needed
    (dict(m=5, a=None, at=None), ARG, "null codes"),
    (dict(sat=None), ARG, "null codes"),
    (dict(out=None), ARG, "null out"),
    (dict(ld=100), ARG, "stride of out"),
    (dict(out=AT["x"]), ARG, "overlaps"),
    (dict(a=AT["x"]), ARG, "overlaps"),
    (dict(at=AT["a"]), ARG, "overlaps"),
    (dict(out=AT["b"], m=4, a=None, at=None), ARG, "overlaps"),
])
def test_linear_refuses(lib, kw, code, why):
    rc, text = linear(lib, **kw)
    assert rc == code and why in text, (rc, text)


def test_linear_needs_memory_for_many_rows_or_large_weights():
    assert not ob.onebit_mx4_linear_needs(4, 4096, 1024)
    assert ob.onebit_mx4_linear_needs(5, 4096, 1024)
    assert ob.onebit_mx4_linear_needs(1, 1 << 15, 1 << 15)
    assert linear(_abi.lib(), m=0, x=None, b=None, sb=None, a=None, at=None, out=None)[0] == 0


def test_linear_binding_refuses_what_is_not_on_the_gpu():
    w = ob.Mx4.empty(40, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        ob.onebit_mx4_linear(torch.zeros(2, 64), w)
    with pytest.raises(TypeError, match="Mx4"):
        ob.onebit_mx4_linear(torch.zeros(2, 64), torch.zeros(40, 64))


def test_everything_raises_without_the_library(monkeypatch):
    w = ob.Mx4.empty(4, 32, device="cpu")
    monkeypatch.setattr(_abi, "LIB_PATH", "/nonexistent/libonebit_adam.so")
    monkeypatch.setattr(_abi, "_lib", None)
    monkeypatch.setattr(ob.adamw, "_native", None)
    x = torch.zeros(4, 32)
    for call in (lambda: ob.onebit_mx4_layout(1, 1), lambda: ob.onebit_mx4_linear_needs(1, 1, 1),
                 lambda: ob.onebit_mx4_quantize(x), lambda: ob.onebit_mx4_dequantize(w),
                 lambda: ob.onebit_mx4_matmul(w, w), lambda: ob.onebit_mx4_linear(x, w),
                 lambda: ob.onebit_mx4_status(0), lambda: ob.Mx4Linear(x)):
        with pytest.raises(RuntimeError, match="not built"):
            call()
