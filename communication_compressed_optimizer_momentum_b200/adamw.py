"""AdamW over a list of tensors: the binding of ``onebit_adamw_*``, ``onebit_adamw8_*`` and
``onebit_grad_norm`` (``include/onebit_adam.h`` has the formulas), and ``AdamW``, which owns the
states of one parameter list.

The functions check every tensor before its address goes to the library: CUDA, contiguous, of the
expected type, length and device. Work is queued on ``stream`` (default: the device's current one)
with the tensors' device current; tensors that are used on another stream than the current one are
marked as used there, so that their memory is not handed out again too early, and results that a
call allocates are that stream's memory. The order between streams is the caller's. The checks are
native (``csrc/binding.cpp``, built into ``_binding.so``): a list may hold hundreds of tensors.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import operator
import os
from typing import List, Sequence, Tuple

from . import _abi

ADAMW_BLOCK = 256
CTL_BYTES = 64
NORM_BYTES = 16384

_native = None


def _binding():
    """The native part of the binding. Raises if it or the library has not been built."""
    global _native
    if _native is None:
        L = _abi.lib()
        import torch  # noqa: F401  (its libraries first)
        again = "`python -m communication_compressed_optimizer_momentum_b200.build`"
        if not os.path.exists(os.path.join(os.path.dirname(__file__), "_binding.so")):
            raise RuntimeError("_binding.so is not built; run " + again)
        try:
            from . import _binding as native
        except ImportError as e:
            raise RuntimeError("_binding.so cannot be loaded (%s); if it is of another Python or "
                               "torch, run %s" % (e, again)) from e
        names = ("onebit_adamw_step", "onebit_adamw8_step", "onebit_adamw8_get_state",
                 "onebit_adamw8_set_state", "onebit_grad_norm",
                 "onebit_internal_adamw_clipped_step")
        native.init({n: ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names},
                    _ob().OneBitError)
        _native = native
    return _native


def _ob():
    import communication_compressed_optimizer_momentum_b200 as ob
    return ob


def _refuse(rc: int, where: str) -> None:
    if rc != 0:
        raise _ob().OneBitError(rc, where, reason=True)


def onebit_adamw_layout(numel: Sequence[int]) -> Tuple[List[int], int]:
    """Where each tensor's part of the flat states begins, and their whole length, in elements."""
    n = len(numel)
    # ctypes would keep the lower 64 bits of a larger number
    lengths = (ctypes.c_int64 * n)(*[x if -1 <= x < 1 << 63 else -1 for x in numel])
    offsets, total = (ctypes.c_int64 * n)(), ctypes.c_int64()
    _refuse(_abi.lib().onebit_adamw_layout(n, lengths, offsets, ctypes.byref(total)),
            "onebit_adamw_layout")
    return list(offsets), total.value


def onebit_adamw_step(params, grads, m, v, ctl, lr, beta1: float = 0.9, beta2: float = 0.999,
                      eps: float = 1e-8, weight_decay=0.0, copies=None, grad_scale=None,
                      bias_correction: bool = True, stream=None) -> None:
    """One AdamW step over a list of tensors with fp32 states, in one launch for up to 800 tensors.

    params, grads: lists of float32 or bfloat16 CUDA tensors (params and grads each of one type),
    any lengths, empty ones too. m, v: flat float32 states of ``onebit_adamw_layout``'s length.
    ctl: int64[8] on the device, zeros before the first step; it counts the steps. lr: a number, or
    a float64 CUDA tensor of one element that is read when the step runs. weight_decay: a number or
    one for each tensor. copies: bfloat16 tensors that receive the new (float32) parameters.
    grad_scale: a float32 CUDA tensor of one element that multiplies every gradient; the step is
    left out if it is not finite."""
    _binding().step("onebit_adamw_step", params, grads, (m, v), ctl, lr, beta1, beta2, eps,
                    weight_decay, copies, grad_scale, bias_correction, stream, None, None, None)


def onebit_adamw8_step(params, grads, m, v, m_exp, v_exp, ctl, lr, beta1: float = 0.9,
                       beta2: float = 0.999, eps: float = 1e-8, weight_decay=0.0, copies=None,
                       grad_scale=None, bias_correction: bool = True, seed: int = 0,
                       stream=None) -> None:
    """``onebit_adamw_step`` with 8-bit states: m, v are uint8 codes of the states' length, m_exp,
    v_exp one uint8 exponent for each 256 of them; all zero for a fresh optimizer. seed selects the
    random bits of the stochastic rounding."""
    _binding().step("onebit_adamw8_step", params, grads, (m, v, m_exp, v_exp), ctl, lr, beta1,
                    beta2, eps, weight_decay, copies, grad_scale, bias_correction, stream, seed,
                    None, None)


def onebit_adamw8_get_state(m, v, m_exp, v_exp, m_out=None, v_out=None, dtype=None, stream=None):
    """What the 8-bit states stand for, as (m, v) of ``dtype`` (float32, the default, or
    bfloat16), allocated unless given."""
    return _binding().get_state8(m, v, m_exp, v_exp, m_out, v_out, dtype, stream)


def onebit_adamw8_set_state(m, v, m_exp, v_exp, m_in, v_in, stream=None) -> None:
    """Encode float32 values of the states' length into the 8-bit states, rounded to nearest. All
    256 values of a block share its exponent: the places behind a tensor have to hold zeros
    (``AdamW.set_state`` sees to that)."""
    _binding().set_state8(m, v, m_exp, v_exp, m_in, v_in, stream)


def onebit_grad_norm(grads, max_norm: float = math.inf, work=None, accumulate: bool = False,
                     stream=None):
    """The l2 norm over a list of gradients and the factor that clips it to ``max_norm``: (norm,
    scale), float32 scalar tensors that stay on the device (views of ``work``; scale is a
    ``grad_scale`` of the steps, NaN if the norm is not finite; the next call with the same work
    overwrites both). work: uint8[16384], zeros before
    its first call; allocated if not given. accumulate: add to the sum of squares in ``work``, for a
    norm over several lists."""
    return _binding().grad_norm(grads, max_norm, work, accumulate, stream)


class AdamW:
    """AdamW of one parameter list: the states (32-bit, or 8-bit with ``state="q8"``), the step
    count and the buffers of the gradient norm.

    ``step(params, grads, lr)`` clips to ``max_norm`` if one is given (one launch for the norm; the
    norm, the factor and the skipping of a step whose norm is not finite stay on the device) and
    updates the tensors in one launch for up to 800 of them. The parameters are the caller's; they are
    passed at every step.

    Every method that reads or writes the states takes a ``stream`` (default: the device's current
    one) and is ordered by it alone: a program that uses several streams makes each wait for the one
    before, first for the one the optimizer was made on. ``counts`` waits for all of them."""

    def __init__(self, params, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay=0.01, max_norm=None, state: str = "f32", seed: int = 0,
                 bias_correction: bool = True):
        import torch
        if state not in ("f32", "q8"):
            raise ValueError("state must be 'f32' or 'q8', got %r" % (state,))
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        if not isinstance(params[0], torch.Tensor):
            raise TypeError("params must be a list of tensors")
        if params[0].dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("params must be float32 or bfloat16, got %s" % params[0].dtype)
        for p in params:
            _ob()._device_vector(p, params[0].dtype, 0, "a parameter", params[0].device)
        self.lengths, self.device = [p.numel() for p in params], params[0].device
        self.beta1, self.beta2, self.eps = beta1, beta2, eps
        self.weight_decay, self.max_norm = weight_decay, max_norm
        self.seed, self.bias_correction = seed, bias_correction
        self.eight = state == "q8"
        self.offsets, self.total = onebit_adamw_layout(self.lengths)

        def zeros(n, dtype):
            return torch.zeros(n, dtype=dtype, device=self.device)

        dtype = torch.uint8 if self.eight else torch.float32
        self.m, self.v = zeros(self.total, dtype), zeros(self.total, dtype)
        if self.eight:
            self.m_exp, self.v_exp = (zeros(self.total // ADAMW_BLOCK, dtype) for _ in range(2))
        self.ctl = zeros(CTL_BYTES // 8, torch.int64)
        self.work = zeros(NORM_BYTES, torch.uint8)

    def step(self, params, grads, lr, copies=None, grad_scale=None, stream=None) -> None:
        _binding().step(
            "onebit_adamw8_step" if self.eight else "onebit_adamw_step", params, grads,
            self._state(), self.ctl, lr, self.beta1, self.beta2, self.eps, self.weight_decay, copies,
            grad_scale, self.bias_correction, stream, self.seed if self.eight else None,
            self.lengths, None if self.max_norm is None else (self.work, self.max_norm))

    @property
    def norm(self):
        """The last step's gradient norm before clipping (with max_norm), on the device: a view that
        the next step overwrites (``clone`` it to keep it)."""
        import torch
        return self.work[8:12].view(torch.float32)[0]

    def counts(self) -> Tuple[int, int]:
        """(steps taken, steps left out); waits for everything that is queued on the device."""
        import torch
        torch.cuda.synchronize(self.device)
        t, skipped = self.ctl[:2].tolist()
        return t, skipped

    def _state(self):
        return (self.m, self.v, self.m_exp, self.v_exp) if self.eight else (self.m, self.v)

    @contextlib.contextmanager
    def _on(self, stream, given=()):
        """``stream`` as the current one, nothing recorded for autograd, and the states and the
        tensors given marked as used there; yields the stream that was current."""
        import torch
        current = torch.cuda.current_stream(self.device)
        if stream is None:
            stream = current
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, self.device) if stream else \
                torch.cuda.default_stream(self.device)
        elif stream.device != self.device:
            raise ValueError("stream is on %s, the states are on %s" % (stream.device, self.device))
        try:
            with torch.cuda.stream(stream), torch.no_grad():
                yield current
        finally:
            if stream != current:
                for x in (*self._state(), self.ctl, *given):
                    if x.is_cuda and x.numel() > 0:
                        x.record_stream(stream)

    def get_state(self, stream=None):
        """Flat float32 (m, v), tensor i at [offsets[i], offsets[i] + lengths[i]): the states
        themselves, or what the 8-bit ones stand for."""
        if not self.eight:
            return self.m, self.v
        return onebit_adamw8_get_state(*self._state(), stream=stream)

    def _encodable(self, x):
        """Flat moments as the 8-bit states take them in: at an aligned address, and zeros behind the
        tensors, whose places share a block's exponent with the tensor's last elements. The caller's
        vector may be a view of any address and hold anything there (a copy of the flat states' size
        where it is, or where any tensor ends within a block)."""
        import torch
        ends = self.offsets[1:] + [self.total]
        gaps = [(o + n, end) for o, n, end in zip(self.offsets, self.lengths, ends) if o + n < end]
        if gaps or x.data_ptr() % 32 != 0:
            x = x.view(-1)[:self.total].clone()
        if gaps:
            torch._foreach_zero_([x[a:b] for a, b in gaps])
        return x

    def set_state(self, m, v, t: int, stream=None) -> None:
        """Continue after step t with these flat float32 moments (8-bit states: rounded). Their
        places behind a tensor may hold anything."""
        import torch
        if t < 0:
            raise ValueError("t must be >= 0")
        for x, name in ((m, "m"), (v, "v")):
            _ob()._device_vector(x, torch.float32, self.total, name, self.device)
        host = torch.zeros(CTL_BYTES // 8, dtype=torch.int64)
        host[0] = t
        host[2:4] = torch.tensor([1.0 - self.beta1 ** t, 1.0 - self.beta2 ** t],
                                 dtype=torch.float64).view(torch.int64)
        with self._on(stream, (m, v)):
            if self.eight:
                onebit_adamw8_set_state(*self._state(), self._encodable(m), self._encodable(v))
            else:
                self.m.copy_(m.view(-1)[:self.total])
                self.v.copy_(v.view(-1)[:self.total])
            self.ctl.copy_(host)                 # last: a call that is refused changes nothing

    def _names(self):
        return ("m", "v", "ctl") + (("m_exp", "v_exp") if self.eight else ())

    def checkpoint(self, stream=None) -> dict:
        """Copies of everything a fresh AdamW of the same list and hyperparameters needs to continue
        bit for bit: states and step count and, of 8-bit states, the seed of the rounding (a CPU
        tensor, so that the whole can be saved or moved like the rest)."""
        import torch
        with self._on(stream) as current:
            ck = {n: getattr(self, n).clone() for n in self._names()}
        for x in ck.values():
            if x.numel() > 0:
                x.record_stream(current)
        if self.eight:
            bits = operator.index(self.seed) & (1 << 64) - 1
            ck["seed"] = torch.tensor(bits - (bits >> 63 << 64), dtype=torch.int64)
        return ck

    def restore(self, ck: dict, stream=None) -> None:
        """Continue from a checkpoint, with its seed (8-bit states; one without a seed leaves the
        optimizer's own). A step that was captured before keeps the seed it was captured with."""
        names = self._names()
        if set(ck) - ({"seed"} if self.eight else set()) != set(names):
            raise ValueError("a checkpoint of another kind of state")
        for n in names:
            own = getattr(self, n)
            if ck[n].dtype != own.dtype or ck[n].shape != own.shape:
                raise ValueError("checkpoint %s has another size or type" % n)
        seed = int(ck["seed"]) if "seed" in ck else self.seed
        with self._on(stream, [ck[n] for n in names]):
            for n in names:
                getattr(self, n).copy_(ck[n])
        self.seed = seed
