"""AdamW over a list of tensors: the binding of ``onebit_adamw_*``, ``onebit_adamw8_*`` and
``onebit_grad_norm`` (``include/onebit_adam.h`` has the formulas), and ``AdamW``, which owns the
states of one parameter list.

The functions check every tensor before its address goes to the library: CUDA, contiguous, of the
expected type, length and device. Work is queued on ``stream`` (default: the device's current one)
with the tensors' device current; tensors that are used on another stream than the current one are
marked as used there, so that their memory is not handed out again too early.
"""
from __future__ import annotations

import ctypes
import math
from operator import attrgetter
from typing import List, Sequence, Tuple

from . import _abi

ADAMW_BLOCK = 256
CTL_BYTES = 64
NORM_BYTES = 16384

_attrs = attrgetter("dtype", "device")


def _ob():
    import communication_compressed_optimizer_momentum_b200 as ob
    return ob


def _refuse(rc: int, where: str) -> None:
    if rc != 0:
        raise _ob().OneBitError(rc, where, reason=True)


def _tensor_list(tensors, name: str, dtype=None, device=None, numel=None):
    """Check a list of tensors of one type on one device; returns (addresses as a C array,
    lengths, type, device)."""
    import torch
    for t in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a list of tensors" % name)
    kinds = set(map(_attrs, tensors))
    if len(kinds) > 1:
        raise ValueError("%s must be of one type on one device, got %s" % (
            name, ", ".join(sorted("%s on %s" % k for k in kinds))))
    for got_dtype, got_device in kinds:
        if got_device.type != "cuda":
            raise ValueError("%s must be CUDA tensors, got device %s" % (name, got_device))
        if device is not None and got_device != device:
            raise ValueError("%s are on %s, expected %s" % (name, got_device, device))
        if dtype is not None and got_dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, got_dtype))
        dtype, device = got_dtype, got_device
    T = torch.Tensor
    if not all(map(T.is_contiguous, tensors)):
        raise ValueError("%s must be contiguous" % name)
    lengths = list(map(T.numel, tensors))
    if numel is not None and lengths != numel:
        raise ValueError("%s have lengths other than the parameters'" % name)
    n = len(lengths)
    return (ctypes.c_void_p * n)(*map(T.data_ptr, tensors)), lengths, dtype, device


def _vector(t, dtype, numel: int, name: str, device):
    _ob()._device_vector(t, dtype, numel, name, device)
    return t.data_ptr()


class _Queue:
    """The device and stream of one call: makes the tensors' device current, and marks tensors as
    used on the stream where that is not the device's current one."""

    def __init__(self, device, stream):
        import torch
        self._guard = torch.cuda.device(device)
        current = torch.cuda.current_stream(device)
        if stream is None:
            stream = current
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else \
                torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError("stream is on %s, the tensors are on %s" % (stream.device, device))
        self._other = stream if stream != current else None
        self.handle = ctypes.c_void_p(stream.cuda_stream)

    def uses(self, *groups) -> None:
        if self._other is None:
            return
        for group in groups:
            for t in group or ():
                if t is not None and t.numel():
                    t.record_stream(self._other)

    def __enter__(self):
        self._guard.__enter__()
        return self

    def __exit__(self, *exc):
        return self._guard.__exit__(*exc)


def _int64s(values):
    return (ctypes.c_int64 * len(values))(*values)


def _dtype_code(dtype, name: str) -> int:
    import torch
    if dtype == torch.float32:
        return 0
    if dtype == torch.bfloat16:
        return 1
    raise TypeError("%s must be float32 or bfloat16, got %s" % (name, dtype))


def onebit_adamw_layout(numel: Sequence[int]) -> Tuple[List[int], int]:
    """Where each tensor's part of the flat states begins, and their whole length, in elements."""
    n = len(numel)
    offsets, total = (ctypes.c_int64 * n)(), ctypes.c_int64()
    _refuse(_abi.lib().onebit_adamw_layout(n, _int64s(list(numel)), offsets, ctypes.byref(total)),
            "onebit_adamw_layout")
    return list(offsets), total.value


def _step(where, params, grads, state, ctl, lr, beta1, beta2, eps, weight_decay, copies,
          grad_scale, bias_correction, stream, seed):
    import torch
    params, grads = list(params), list(grads)
    if len(grads) != len(params):
        raise ValueError("%d gradients for %d parameters" % (len(grads), len(params)))
    _ob()._device_vector(ctl, torch.int64, CTL_BYTES // 8, "ctl")
    device = ctl.device
    p, lengths, ptype, _ = _tensor_list(params, "params", device=device)
    g, _, gtype, _ = _tensor_list(grads, "grads", device=device, numel=lengths)
    ptype = _dtype_code(ptype, "params") if params else 0
    gtype = _dtype_code(gtype, "grads") if grads else 0
    c = None
    if copies is not None:
        copies = list(copies)
        if len(copies) != len(params):
            raise ValueError("%d copies for %d parameters" % (len(copies), len(params)))
        c = _tensor_list(copies, "copies", torch.bfloat16, device, lengths)[0]
    total = sum([-(-n // ADAMW_BLOCK) for n in lengths]) * ADAMW_BLOCK
    pointers = [_vector(t, torch.uint8 if seed is not None else torch.float32,
                        total // ADAMW_BLOCK if name.endswith("_exp") else total, name, device)
                for name, t in state]
    if isinstance(weight_decay, (int, float)):
        weight_decay = [weight_decay] * len(params)
    if len(weight_decay) != len(params):
        raise ValueError("%d weight decays for %d parameters" % (len(weight_decay), len(params)))
    wd = (ctypes.c_double * len(params))(*weight_decay)
    scale = None if grad_scale is None else _vector(grad_scale, torch.float32, 1, "grad_scale",
                                                    device)
    lr_dev = None
    if isinstance(lr, torch.Tensor):
        lr_dev, lr_tensor, lr = _vector(lr, torch.float64, 1, "lr", device), lr, 0.0
    else:
        lr_tensor = None
    args = [len(params), _int64s(lengths), p, ptype, g, gtype, c, *pointers, ctl.data_ptr()]
    if seed is not None:
        args.append(int(seed) & 0xFFFFFFFFFFFFFFFF)
    with _Queue(device, stream) as q:
        rc = getattr(_abi.lib(), where)(*args, wd, scale, lr_dev, lr, beta1, beta2, eps,
                                        1 if bias_correction else 0, q.handle)
        _refuse(rc, where)
        q.uses(params, grads, copies, [t for _, t in state], [ctl, grad_scale, lr_tensor])


def onebit_adamw_step(params, grads, m, v, ctl, lr, beta1: float = 0.9, beta2: float = 0.999,
                      eps: float = 1e-8, weight_decay=0.0, copies=None, grad_scale=None,
                      bias_correction: bool = True, stream=None) -> None:
    """One AdamW step over a list of tensors with fp32 states, in one launch.

    params, grads: lists of float32 or bfloat16 CUDA tensors (params and grads each of one type),
    any lengths, empty ones too. m, v: flat float32 states of ``onebit_adamw_layout``'s length.
    ctl: int64[8] on the device, zeros before the first step; it counts the steps. lr: a number, or
    a float64 CUDA tensor of one element that is read when the step runs. weight_decay: a number or
    one for each tensor. copies: bfloat16 tensors that receive the new (float32) parameters.
    grad_scale: a float32 CUDA tensor of one element that multiplies every gradient; the step is
    left out if it is not finite."""
    _step("onebit_adamw_step", params, grads, (("m", m), ("v", v)), ctl, lr, beta1, beta2, eps,
          weight_decay, copies, grad_scale, bias_correction, stream, None)


def onebit_adamw8_step(params, grads, m, v, m_exp, v_exp, ctl, lr, beta1: float = 0.9,
                       beta2: float = 0.999, eps: float = 1e-8, weight_decay=0.0, copies=None,
                       grad_scale=None, bias_correction: bool = True, seed: int = 0,
                       stream=None) -> None:
    """``onebit_adamw_step`` with 8-bit states: m, v are uint8 codes of the states' length, m_exp,
    v_exp one uint8 exponent for each 256 of them; all zero for a fresh optimizer. seed selects the
    random bits of the stochastic rounding."""
    _step("onebit_adamw8_step", params, grads,
          (("m", m), ("v", v), ("m_exp", m_exp), ("v_exp", v_exp)), ctl, lr, beta1, beta2, eps,
          weight_decay, copies, grad_scale, bias_correction, stream, seed)


def _state8(m, v, m_exp, v_exp):
    import torch
    _ob()._device_vector(m, torch.uint8, 0, "m")
    total = m.numel()
    if total % ADAMW_BLOCK:
        raise ValueError("m holds %d codes, not a multiple of %d" % (total, ADAMW_BLOCK))
    for t, n, name in ((v, total, "v"), (m_exp, total // ADAMW_BLOCK, "m_exp"),
                       (v_exp, total // ADAMW_BLOCK, "v_exp")):
        _vector(t, torch.uint8, n, name, m.device)
    return total, m.device


def onebit_adamw8_get_state(m, v, m_exp, v_exp, m_out=None, v_out=None, dtype=None, stream=None):
    """What the 8-bit states stand for, as (m, v) of ``dtype`` (float32, the default, or
    bfloat16), allocated unless given."""
    import torch
    total, device = _state8(m, v, m_exp, v_exp)
    given = next((t.dtype for t in (m_out, v_out) if t is not None), None)
    dtype = dtype or given or torch.float32
    code = _dtype_code(dtype, "the values")
    with _Queue(device, stream) as q:
        if m_out is None:
            m_out = torch.empty(total, dtype=dtype, device=device)
        if v_out is None:
            v_out = torch.empty(total, dtype=dtype, device=device)
        args = [_vector(m_out, dtype, total, "m_out", device),
                _vector(v_out, dtype, total, "v_out", device)]
        _refuse(_abi.lib().onebit_adamw8_get_state(
            total, m.data_ptr(), v.data_ptr(), m_exp.data_ptr(), v_exp.data_ptr(), *args, code,
            q.handle), "onebit_adamw8_get_state")
        q.uses((m, v, m_exp, v_exp, m_out, v_out))
    return m_out, v_out


def onebit_adamw8_set_state(m, v, m_exp, v_exp, m_in, v_in, stream=None) -> None:
    """Encode float32 values of the states' length into the 8-bit states, rounded to nearest."""
    import torch
    total, device = _state8(m, v, m_exp, v_exp)
    args = [_vector(m_in, torch.float32, total, "m_in", device),
            _vector(v_in, torch.float32, total, "v_in", device)]
    with _Queue(device, stream) as q:
        _refuse(_abi.lib().onebit_adamw8_set_state(
            total, m.data_ptr(), v.data_ptr(), m_exp.data_ptr(), v_exp.data_ptr(), *args,
            q.handle), "onebit_adamw8_set_state")
        q.uses((m, v, m_exp, v_exp, m_in, v_in))


def onebit_grad_norm(grads, max_norm: float = math.inf, work=None, accumulate: bool = False,
                     stream=None):
    """The l2 norm over a list of gradients and the factor that clips it to ``max_norm``: (norm,
    scale), float32 scalar tensors that stay on the device (views of ``work``; scale is a
    ``grad_scale`` of the steps, NaN if the norm is not finite). work: uint8[16384], zeros before
    its first call; allocated if not given. accumulate: add to the sum of squares in ``work``, for a
    norm over several lists."""
    import torch
    grads = list(grads)
    if work is None:
        if accumulate:
            raise ValueError("accumulate needs the work of the first call")
        if not grads:
            raise ValueError("no gradients and no work to say where")
        device = _tensor_list(grads, "grads")[3]
        with _Queue(device, stream) as q, torch.cuda.stream(q._other):
            work = torch.zeros(NORM_BYTES, dtype=torch.uint8, device=device)
    _ob()._device_vector(work, torch.uint8, NORM_BYTES, "work")
    g, lengths, gtype, _ = _tensor_list(grads, "grads", device=work.device)
    gtype = _dtype_code(gtype, "grads") if grads else 0
    with _Queue(work.device, stream) as q:
        _refuse(_abi.lib().onebit_grad_norm(
            len(grads), _int64s(lengths), g, gtype, max_norm, 1 if accumulate else 0,
            work.data_ptr(), q.handle), "onebit_grad_norm")
        q.uses(grads, (work,))
    return work[8:16].view(torch.float32).unbind()


class AdamW:
    """AdamW of one parameter list: the states (32-bit, or 8-bit with ``state="q8"``), the step
    count and the buffers of the gradient norm.

    ``step(params, grads, lr)`` clips to ``max_norm`` if one is given (the norm, the factor and the
    skipping of a step whose norm is not finite stay on the device) and updates every tensor in one
    launch. The parameters are the caller's; they are passed at every step."""

    def __init__(self, params, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay=0.01, max_norm=None, state: str = "f32", seed: int = 0,
                 bias_correction: bool = True):
        import torch
        if state not in ("f32", "q8"):
            raise ValueError("state must be 'f32' or 'q8', got %r" % (state,))
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        _, self.lengths, _, self.device = _tensor_list(params, "params")
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
        params, grads = list(params), list(grads)
        if [p.numel() for p in params] != self.lengths:
            raise ValueError("params have lengths other than the optimizer's")
        if self.max_norm is not None:
            if grad_scale is not None:
                raise ValueError("grad_scale and max_norm exclude each other")
            grad_scale = onebit_grad_norm(grads, self.max_norm, self.work, stream=stream)[1]
        kw = dict(copies=copies, grad_scale=grad_scale, bias_correction=self.bias_correction,
                  stream=stream)
        args = (self.ctl, lr, self.beta1, self.beta2, self.eps, self.weight_decay)
        if self.eight:
            onebit_adamw8_step(params, grads, self.m, self.v, self.m_exp, self.v_exp, *args,
                               seed=self.seed, **kw)
        else:
            onebit_adamw_step(params, grads, self.m, self.v, *args, **kw)

    @property
    def norm(self):
        """The last step's gradient norm before clipping (with max_norm), on the device."""
        import torch
        return self.work[8:12].view(torch.float32)[0]

    def counts(self) -> Tuple[int, int]:
        """(steps taken, steps left out); waits for the device."""
        t, skipped = self.ctl[:2].tolist()
        return t, skipped

    def _state(self):
        return (self.m, self.v, self.m_exp, self.v_exp)

    def get_state(self, stream=None):
        """Flat float32 (m, v), tensor i at [offsets[i], offsets[i] + lengths[i]): the states
        themselves, or what the 8-bit ones stand for."""
        if not self.eight:
            return self.m, self.v
        return onebit_adamw8_get_state(*self._state(), stream=stream)

    def set_state(self, m, v, t: int, stream=None) -> None:
        """Continue after step t with these flat float32 moments (8-bit states: rounded)."""
        import torch
        if t < 0:
            raise ValueError("t must be >= 0")
        _vector(m, torch.float32, self.total, "m", self.device)
        _vector(v, torch.float32, self.total, "v", self.device)
        host = torch.zeros(CTL_BYTES // 8, dtype=torch.int64)
        host[0] = t
        host[2:4] = torch.tensor([1.0 - self.beta1 ** t, 1.0 - self.beta2 ** t],
                                 dtype=torch.float64).view(torch.int64)
        with _Queue(self.device, stream) as q, torch.cuda.stream(q._other):
            self.ctl.copy_(host)
            if not self.eight:
                self.m.copy_(m[:self.total])
                self.v.copy_(v[:self.total])
        if self.eight:
            onebit_adamw8_set_state(*self._state(), m, v, stream=stream)

    def checkpoint(self) -> dict:
        """Copies of everything a fresh AdamW of the same list needs to continue bit for bit."""
        names = ("m", "v", "ctl") + (("m_exp", "v_exp") if self.eight else ())
        return {n: getattr(self, n).clone() for n in names}

    def restore(self, ck: dict) -> None:
        names = ("m", "v", "ctl") + (("m_exp", "v_exp") if self.eight else ())
        if set(ck) != set(names):
            raise ValueError("a checkpoint of another kind of state")
        for n in names:
            own = getattr(self, n)
            if ck[n].dtype != own.dtype or ck[n].shape != own.shape:
                raise ValueError("checkpoint %s has another size or type" % n)
        for n in names:
            getattr(self, n).copy_(ck[n])
