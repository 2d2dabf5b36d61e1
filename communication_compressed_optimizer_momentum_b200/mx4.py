"""Matrices in microscaled 4-bit floating point: the binding of ``onebit_mx4_*``
(``include/onebit_adam.h`` has the format and the formulas), and ``Mx4Linear``, the passes of a
linear layer whose weights, activations and gradients are multiplied in 4 bits.

Tensors are checked before their addresses go to the library. Work is queued on ``stream`` (default:
the device's current one) with the tensors' device current; tensors that are used on another stream
than the current one are marked as used there, and results that a call allocates are that stream's
memory. The order between streams is the caller's. Nothing is recorded for autograd.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

from . import _abi
from .adamw import _binding, _refuse

MX4_BLOCK = 32
_FORMS = {"rows": (True, False), "columns": (False, True), "both": (True, True)}
_ROUNDINGS = {"nearest": False, "stochastic": True}


def onebit_mx4_layout(rows: int, cols: int) -> Tuple[int, int]:
    """The lengths of a matrix's codes and scales, in bytes."""
    size = [ctypes.c_int64(x if -1 <= x < 1 << 63 else -1) for x in (rows, cols)]
    codes, scales = ctypes.c_int64(), ctypes.c_int64()
    _refuse(_abi.lib().onebit_mx4_layout(*size, ctypes.byref(codes), ctypes.byref(scales)),
            "onebit_mx4_layout")
    return codes.value, scales.value


class Mx4:
    """A matrix of rows x cols in 4 bits, in the library's layout: ``codes`` and ``scales``, uint8 CUDA
    tensors. Blocks of 32 consecutive columns share an exponent."""

    __slots__ = ("_codes", "_scales", "rows", "cols")

    def __init__(self, codes, scales, rows: int, cols: int):
        # scales None: codes holds both, one after the other
        self._codes, self._scales, self.rows, self.cols = codes, scales, rows, cols

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "Mx4":
        """Room for a matrix, to be an ``out``."""
        import torch
        return cls(torch.empty(sum(onebit_mx4_layout(rows, cols)), dtype=torch.uint8, device=device),
                   None, rows, cols)

    @property
    def codes(self):
        """[rows][bytes of a row], two codes a byte."""
        n = onebit_mx4_layout(self.rows, self.cols)[0]
        return self._codes.view(-1)[:n].view(self.rows, n // self.rows if self.rows else 0)

    @property
    def scales(self):
        """The blocks' exponents, in tiles of 128 rows by four blocks."""
        n, m = onebit_mx4_layout(self.rows, self.cols)
        return self._codes.view(-1)[n:n + m] if self._scales is None else self._scales

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self):
        return self._codes.device

    def _parts(self):
        return self._codes, self._scales, self.rows, self.cols

    def __repr__(self):
        return "Mx4(%d x %d, %s)" % (self.rows, self.cols, self.device)


def _parts(q, name: str):
    if not isinstance(q, Mx4):
        raise TypeError("%s must be an Mx4, got %s" % (name, type(q).__name__))
    return q._parts()


def _one_of(table, value, name: str):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError("%s must be one of %s, got %r" % (name, ", ".join(map(repr, table)), value)
                         ) from None


def onebit_mx4_quantize(x, forms: str = "rows", rounding: str = "nearest", seed: int = 0,
                        residual=None, out=None, stream=None):
    """Quantise a float32 or bfloat16 CUDA matrix (consecutive columns, rows that do not overlap at any
    distance; faster where all of them begin at multiples of 32 bytes).

    forms: "rows" gives the matrix, in blocks of 32 of a row; "columns" its transpose, in blocks of
    32 of a column; "both" the pair (matrix, transpose) from one pass over x. rounding: "nearest", or
    "stochastic" with the random bits of seed (and seed + 1 for the transpose: seeds of calls whose errors
    are to be unrelated are two or more apart). residual (a float32
    matrix of x's size, with forms="rows"): error feedback; x + residual is quantised, and residual
    becomes what that lost. out: an ``Mx4`` (with "both" a pair) to write to, else new ones."""
    rows, columns = _one_of(_FORMS, forms, "forms")
    stochastic = _one_of(_ROUNDINGS, rounding, "rounding")
    if residual is not None and forms != "rows":
        raise ValueError("a residual goes with forms='rows'")
    to_rows = to_columns = None
    if out is not None:
        if forms == "both":
            to_rows, to_columns = (_parts(q, "out") for q in out)
        elif rows:
            to_rows = _parts(out, "out")
        else:
            to_columns = _parts(out, "out")
    own, transposed = _binding().mx4_quantize(x, rows, columns, stochastic, seed, residual, to_rows,
                                              to_columns, stream)
    if out is not None:
        return out
    r, c = x.shape
    if not columns:
        return Mx4(own, None, r, c)
    if not rows:
        return Mx4(transposed, None, c, r)
    return Mx4(own, None, r, c), Mx4(transposed, None, c, r)


def onebit_mx4_dequantize(q, dtype=None, out=None, stream=None):
    """What an ``Mx4`` stands for, as a matrix of ``dtype`` (float32, the default, or bfloat16; exact
    in both), allocated unless given."""
    return _binding().mx4_dequantize(_parts(q, "q"), dtype, out, stream)


def onebit_mx4_matmul(a, b, out=None, dtype=None, accumulate: bool = False, stream=None):
    """a b^T of two ``Mx4`` matrices of as many columns, float32 sums; bfloat16 (the default) or
    float32, allocated unless given (consecutive columns, rows that do not overlap at any distance; faster
    where all of them begin at multiples of 16 bytes). accumulate: added to a float32 out."""
    return _binding().mx4_matmul(_parts(a, "a"), _parts(b, "b"), out, dtype, accumulate, stream)


def onebit_mx4_linear(x, w, keep: bool = False, dtype=None, stream=None):
    """q(x) w^T for x [..., inner] (float32 or bfloat16, rounded to nearest) and an ``Mx4`` w of inner
    columns, of ``dtype`` (x's by default). keep: the pair with x in 4 bits in blocks along its rows, as
    ``onebit_mx4_quantize(x, forms="columns")`` gives it."""
    if not keep:
        return _binding().mx4_forward(x, _parts(w, "w"), False, dtype, stream)
    y, kept = _binding().mx4_forward(x, _parts(w, "w"), True, dtype, stream)
    return y, Mx4(kept, None, w.cols, x.shape[:-1].numel())


def onebit_mx4_linear_needs(m: int, n: int, k: int) -> bool:
    """Whether ``onebit_mx4_linear`` of these sizes needs memory for x in 4 bits."""
    return bool(_abi.lib().onebit_mx4_linear_needs(m, n, k))


def onebit_mx4_status(stream=None) -> int:
    """Not 0 if a wait within a product on the current device ever gave up. Waits for the stream."""
    from . import _stream
    flags = ctypes.c_uint32()
    _refuse(_abi.lib().onebit_mx4_status(ctypes.byref(flags), _stream(stream)), "onebit_mx4_status")
    return flags.value


class Mx4Linear:
    """A linear layer's weights in 4 bits, and its passes: y = x W^T, dx = dy W, dW = dy^T x, each a
    product of two 4-bit matrices with float32 sums.

    The weights are held in blocks of 32 along both axes (``w`` for the forward product, ``wt`` for
    the backward one; without ``backward`` only the first). ``update`` quantises them again into the
    same memory, so that captured passes stay valid: after every optimizer step, or through
    ``AdamW.step(..., mx4=[...])``. Activations and weights are rounded to nearest, gradients
    stochastically, so that the weights' gradients keep their means."""

    def __init__(self, weight, backward: bool = True, stream=None):
        import torch
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
            raise TypeError("weight must be a matrix [outer][inner]")
        self.outer, self.inner = weight.shape
        q = onebit_mx4_quantize(weight.detach(), forms="both" if backward else "rows", stream=stream)
        self.w, self.wt = q if backward else (q, None)

    @property
    def device(self):
        return self.w.device

    def check_weight(self, weight) -> None:
        """Raises unless ``update`` would take this weight."""
        import torch
        if not isinstance(weight, torch.Tensor) or tuple(weight.shape) != (self.outer, self.inner):
            raise ValueError("weight must be a matrix of %d x %d" % (self.outer, self.inner))
        if weight.device != self.device:
            raise ValueError("weight is on %s, expected %s" % (weight.device, self.device))
        if weight.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("weight must be float32 or bfloat16, got %s" % weight.dtype)
        if weight.is_contiguous():
            return
        rows, cols = weight.stride()
        if self.inner > 1 and cols != 1:
            raise ValueError("weight must have consecutive columns")
        if self.outer > 1 and self.inner > 0 and rows < self.inner:
            raise ValueError("weight must have rows of its own: they are %d apart" % rows)

    def update(self, weight, stream=None) -> None:
        """Quantise the weights anew."""
        self.check_weight(weight)
        if self.wt is None:
            onebit_mx4_quantize(weight.detach(), out=self.w, stream=stream)
        else:
            onebit_mx4_quantize(weight.detach(), forms="both", out=(self.w, self.wt), stream=stream)

    def forward(self, x, keep: bool = False, dtype=None, stream=None):
        """y = x W^T for x [..., inner] (float32 or bfloat16), of ``dtype`` (x's by default). keep:
        (y, kept), where kept is x in 4 bits in blocks along the tokens, what ``backward`` needs."""
        return onebit_mx4_linear(x, self.w, keep, dtype, stream)

    def backward(self, dy, kept: Optional[Mx4] = None, seed: int = 0, grad=None,
                 accumulate: bool = False, dtype=None, need_dx: bool = True, stream=None):
        """(dx, dW) for dy [..., outer]. dx is of ``dtype`` (dy's by default), None without need_dx.
        dW comes from what ``forward`` kept (without it None): a float32 matrix, or into grad (float32
        or bfloat16), added to it with accumulate (float32). seed selects the random bits that dy is
        rounded with, those of seed for dx and of seed + 1 for dW: every call of every layer and step takes
        one of its own, two or more from all others (2 * (step * layers + layer), say). With the same or
        the next number every value still keeps its mean, but calls share their errors place by place."""
        if kept is None and (grad is not None or accumulate):
            raise ValueError("grad and accumulate need what forward kept")
        if accumulate and grad is None:
            raise ValueError("accumulate needs grad")
        if need_dx and self.wt is None:
            raise ValueError("made without backward=True: dx needs the weights along the outer axis")
        if not need_dx and kept is None:
            return None, None
        return _binding().mx4_backward(
            dy, self.wt._parts() if need_dx else None, None if kept is None else _parts(kept, "kept"),
            self.outer, self.inner, seed, grad, accumulate, dtype, stream)
