"""The optimizer step (``include/fp8q_adamw.h``): the binding of
``adamw_step``. Imported by the package; see its docstring."""
from __future__ import annotations

import ctypes

import torch

from . import Fp8qError, _check, _load
from ._mx4 import _address, _call, _on_gpu

ADAMW_BF16 = 0
ADAMW_F32 = 1

_DTYPES = {torch.bfloat16: ADAMW_BF16, torch.float32: ADAMW_F32}
_CODES = (torch.float8_e4m3fn, torch.uint8)

_lib = None


class _Tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("numel", ctypes.c_int64)]


def _library():
    """The C library with the signature of the optimizer's entry point."""
    global _lib
    if _lib is None:
        L = _load()
        p, i64, i32, cint, f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_double
        L.adamw_step.argtypes = [i32, p, p, cint, cint, cint, f64, f64, f64, f64, f64, i64, p, p, p, ctypes.c_uint64, p]
        L.adamw_step.restype = cint
        _lib = L
    return _lib


class AdamwPlan:
    """The tensors of an optimizer, checked once by :func:`adamw_plan`. It keeps
    their storage alive and steps what is there: after a tensor has been given
    other storage, make a new plan. One thread at a time steps a plan."""

    __slots__ = ("device", "shapes", "param_dtype", "state_bits", "_entries", "_tensors", "_grads")

    def __init__(self, device, shapes, param_dtype, state_bits, entries, tensors):
        self.device, self.shapes, self.param_dtype, self.state_bits = device, shapes, param_dtype, state_bits
        self._entries, self._tensors = entries, tensors
        self._grads = (ctypes.c_void_p * len(shapes))()

    def __len__(self):
        return len(self.shapes)


def _same_list(ts, count: int, what: str):
    ts = list(ts)
    if len(ts) != count:
        raise Fp8qError("%s has %d tensors, params has %d" % (what, len(ts), count))
    return ts


def _array(t: torch.Tensor, shape, dtypes, what: str, i: int) -> None:
    if t.dtype not in dtypes:
        raise Fp8qError("%s[%d] has dtype %s, expected %s" % (what, i, t.dtype, " or ".join(str(d) for d in dtypes)))
    if t.shape != shape:
        raise Fp8qError("%s[%d] has shape %s, expected %s" % (what, i, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise Fp8qError("%s[%d] must be contiguous" % (what, i))


def _overlaps(ts) -> bool:
    """Whether two of the tensors share memory."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in ts if t.numel() > 0)
    return any(a[1] > b[0] for a, b in zip(spans, spans[1:]))


def adamw_plan(params, exp_avg, exp_avg_sq, exp_avg_scale=None, exp_avg_sq_scale=None, copies=None) -> AdamwPlan:
    """The tensors that :func:`adamw_step` updates, looked over once.

    ``params``: FP32 or bf16 tensors (all of one dtype), contiguous, of any
    number and shape, up to 2^34 - 1024 elements each. ``exp_avg``, ``exp_avg_sq``: states of the same shapes,
    zero at the start of training: FP32, or E4M3 codes (``float8_e4m3fn`` or
    uint8) for states in 8 bits, where ``exp_avg_sq`` holds the ROOT of the
    second moment and ``exp_avg_scale``, ``exp_avg_sq_scale`` are FP32
    ``[ceil(numel / 128)]`` for each tensor, one scale for 128 consecutive
    elements. ``copies``: bf16 tensors of the same shapes (None for a tensor
    without one) that every step writes the new FP32 parameters to.
    """
    params = list(params)
    count = len(params)
    avg, sq = _same_list(exp_avg, count, "exp_avg"), _same_list(exp_avg_sq, count, "exp_avg_sq")
    if (exp_avg_scale is None) != (exp_avg_sq_scale is None):
        raise Fp8qError("states in 8 bits need the scales of both moments")
    bits = 32 if exp_avg_scale is None else 8
    none = [None] * count
    avg_s = none if bits == 32 else _same_list(exp_avg_scale, count, "exp_avg_scale")
    sq_s = none if bits == 32 else _same_list(exp_avg_sq_scale, count, "exp_avg_sq_scale")
    copies = none if copies is None else _same_list(copies, count, "copies")
    every = [t for ts in (params, avg, sq, avg_s, sq_s, copies) for t in ts if t is not None]
    device = _on_gpu(*every)
    dtype = params[0].dtype if count else torch.float32
    if dtype not in _DTYPES:
        raise Fp8qError("params must be float32 or bfloat16, got %s" % dtype)
    states = (torch.float32,) if bits == 32 else _CODES
    entries = (_Tensor * max(count, 1))()
    for i, p in enumerate(params):
        shape = p.shape
        _array(p, shape, (dtype,), "params", i)
        _array(avg[i], shape, states, "exp_avg", i)
        _array(sq[i], shape, states, "exp_avg_sq", i)
        if bits == 8:
            blocks = torch.Size((-(-p.numel() // 128),))
            _array(avg_s[i], blocks, (torch.float32,), "exp_avg_scale", i)
            _array(sq_s[i], blocks, (torch.float32,), "exp_avg_sq_scale", i)
        if copies[i] is not None:
            if dtype is not torch.float32:
                raise Fp8qError("copies belong to float32 params")
            _array(copies[i], shape, (torch.bfloat16,), "copies", i)
        entries[i] = _Tensor(p.data_ptr(), avg[i].data_ptr(), sq[i].data_ptr(), _address(avg_s[i]),
                             _address(sq_s[i]), _address(copies[i]), p.numel())
    if _overlaps(every):
        raise Fp8qError("two of the plan's tensors share memory")
    # (views of their own: a parameter that is given other storage leaves this one to the plan)
    return AdamwPlan(device, [p.shape for p in params], dtype, bits, entries, [t.detach() for t in every])


_dtype_of, _shape_of = torch.Tensor.dtype.__get__, torch.Tensor.shape.__get__
_is_contiguous, _device_of, _address_of = torch.Tensor.is_contiguous, torch.Tensor.get_device, torch.Tensor.data_ptr


def _gradients(plan: AdamwPlan, grads):
    """Checks the gradients, puts their addresses into the plan's array and returns their dtype (None: there is none)."""
    shapes, there = plan.shapes, grads
    if type(None) in set(map(type, grads)):
        there = [g for g in grads if g is not None]
        shapes = [s for s, g in zip(shapes, grads) if g is not None]
    if not there:
        return None
    dtype, device = there[0].dtype, plan.device
    if dtype not in _DTYPES:
        raise Fp8qError("grads must be float32 or bfloat16, got %s" % dtype)
    # (whole lists at a time: a step of many small tensors takes the GPU less than a look at each of them takes here)
    if (list(map(_shape_of, there)) != shapes or set(map(_dtype_of, there)) != {dtype}
            or not all(map(_is_contiguous, there)) or set(map(_device_of, there)) != {device}):
        for i, g in enumerate(grads):
            if g is not None:
                _array(g, plan.shapes[i], (dtype,), "grads", i)
                if g.get_device() != device:
                    raise Fp8qError("grads[%d] must live on cuda:%d" % (i, device))
    if there is grads:
        plan._grads[:] = list(map(_address_of, grads))
    else:
        plan._grads[:] = [None if g is None else g.data_ptr() for g in grads]
    return dtype


def _one(t: torch.Tensor, dtype, name: str) -> int:
    if t.dtype is not dtype or t.numel() != 1:
        raise Fp8qError("%s must hold one %s element" % (name, dtype))
    return t.data_ptr()


def adamw_step(plan: AdamwPlan, grads, step, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.01, grad_scale: torch.Tensor | None = None, seed: int = 0,
               stream=None) -> None:
    """One AdamW step of a plan's tensors, in place:
    ``m = beta1 m + (1 - beta1) g``, ``v = beta2 v + (1 - beta2) g^2``,
    ``p = p (1 - lr weight_decay) - lr / (1 - beta1^step) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)``,
    one launch for each 64 tensors (56 with 8-bit states).

    ``grads``: bf16 or FP32 tensors (all of one dtype), contiguous, of the
    params' shapes, sharing no memory with the plan's tensors; None leaves a
    tensor as it is. ``step``: 1 in the first
    step; ``step`` and ``lr`` are numbers, or GPU tensors of one element (int64,
    float32) that are read when the step runs, as a captured step that is
    replayed needs. ``grad_scale``: a GPU tensor of one float32 element that the
    gradients are multiplied with (clipping, loss scaling); where it is not
    finite, nothing is changed. ``seed`` chooses the random bits with which
    states in 8 bits are rounded; they differ from step to step by themselves.

    As everywhere in this package there is no autograd, and the tensors are
    changed behind its back.
    """
    grads = _same_list(grads, len(plan), "grads")
    dtype = _gradients(plan, grads)
    if dtype is None:
        return
    device = plan.device
    on_gpu = [t for t in (grad_scale, step, lr) if torch.is_tensor(t)]
    if on_gpu and _on_gpu(*on_gpu) != device:
        raise Fp8qError("step, lr and grad_scale must live on cuda:%d" % device)
    lr_dev = step_dev = 0
    if torch.is_tensor(lr):
        lr, lr_dev = 0.0, _one(lr, torch.float32, "lr")
    if torch.is_tensor(step):
        step, step_dev = 1, _one(step, torch.int64, "step")
    elif not 1 <= step <= 0x7FFFFFFFFFFFFFFF:
        raise Fp8qError("step must be at least 1, got %d" % step)
    if not 0 <= seed < 1 << 64:
        raise Fp8qError("seed must be within 64 bits, got %d" % seed)
    scale = 0 if grad_scale is None else _one(grad_scale, torch.float32, "grad_scale")
    st = _call(_library().adamw_step, device, stream, len(grads), plan._entries, plan._grads, _DTYPES[plan.param_dtype], _DTYPES[dtype],
               plan.state_bits, lr, beta1, beta2, eps, weight_decay, int(step), lr_dev, step_dev, scale, seed)
    _check(st, "adamw_step")
