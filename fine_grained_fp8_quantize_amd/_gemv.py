"""Products of few bf16 rows with FP4 weights (``include/fp8q_gemv.h``): the
binding of ``fp4_gemv_mx`` and ``fp4_gated_gemv_mx``. Imported by the package;
see its docstring."""
from __future__ import annotations

import ctypes

import torch

from . import Fp8qError, _check, _load, _out_code
from ._gated import _act_code
from ._mx4 import _address, _call, _matrix, _new, _on_gpu, _rows_of, _tiles_ld

_WORDS = (torch.int32, torch.uint32)

_lib = None


def _library():
    """The C library with the signatures of the weight-only entry points."""
    global _lib
    if _lib is None:
        L = _load()
        p, i64, i32, cint = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
        L.fp4_gemv_mx.argtypes = [i64, i32, p, i32, i32, i64, i64, p, i64, i64, p, i64, i64, p, i64, i64, p, i64, cint, p]
        L.fp4_gated_gemv_mx.argtypes = [i64, i32, p, i32, i32, i64, i64, p, i64, i64, p, i64, i64, i64, p, i64, i64, i64,
                                        cint, p, i64, cint, p]
        L.fp4_gemv_mx.restype = L.fp4_gated_gemv_mx.restype = cint
        _lib = L
    return _lib


def _weights(w: torch.Tensor, w_scale: torch.Tensor, lead: int):
    """K tiles, row tiles, leading dimensions and strides of FP4 weights with ``lead`` dimensions of stacked matrices."""
    qs, ss = w.shape, w_scale.shape
    if (w.dtype is torch.uint8 and w_scale.dtype is torch.int32 and len(qs) == 3 + lead and qs[-1] == 1024
            and w.is_contiguous() and w_scale.is_contiguous()):
        kt, rt = qs[-3], qs[-2]
        if ss[lead:] == ((kt + 3) // 4, rt, 64) and ss[:lead] == qs[:lead]:  # the usual case, in few steps
            return kt, rt, rt, rt, w.stride(), w_scale.stride()
    if lead < 2:
        return (*_matrix(w, w_scale, "w", lead), w.stride(), w_scale.stride())
    if w.dtype is not torch.uint8 or len(qs) != 5 or qs[-1] != 1024:
        raise Fp8qError("w must be uint8 [E][2][k tiles][row tiles][1024]")
    kt, rt = qs[-3], qs[-2]
    if w_scale.dtype not in _WORDS or ss != (*qs[:2], (kt + 3) // 4, rt, 64):
        raise Fp8qError("w_scale must be int32 %s, got %s %s" % ((*qs[:2], (kt + 3) // 4, rt, 64), w_scale.dtype,
                                                                 tuple(ss)))
    return kt, rt, _tiles_ld(w, 1024, lead, "w"), _tiles_ld(w_scale, 64, lead, "w_scale"), w.stride(), w_scale.stride()


def _gemv(x, w, w_scale, n, ids, first, gated, act, out_dtype, out, stream, name):
    dev = _on_gpu(x, w, w_scale, ids, out)
    if x.dtype is not torch.bfloat16:
        raise Fp8qError("x must be bfloat16")
    routed = 0 if ids is None else 1
    kt, rt, ld_w, ld_s, w_strides, s_strides = _weights(w, w_scale, routed + 1 if gated else routed)
    if gated and w.shape[routed] != 2:
        raise Fp8qError("gated weights are stacked in twos, gate first; got %d" % w.shape[routed])
    n = _rows_of(n, rt, "n")
    xs = x.shape
    k = xs[-1] if xs else 0
    if routed:
        if ids.dtype is not torch.int32 or ids.dim() != 2 or not ids.is_contiguous():
            raise Fp8qError("ids must be a contiguous int32 [tokens][topk] tensor")
        tokens, topk = ids.shape
        experts = w.shape[0]
        if not 0 <= first <= 0x7FFFFFFF - experts:
            raise Fp8qError("first = %d is out of range" % first)
        if len(xs) not in (2, 3) or xs[0] != tokens or (len(xs) == 3 and xs[1] != topk):
            raise Fp8qError("x must be [tokens][k] or [tokens][topk][k] for ids %s, got %s" % (tuple(ids.shape), tuple(xs)))
        shape, stride_w, stride_s = (tokens, topk, n), w_strides[0], s_strides[0]
    else:
        if len(xs) != 2:
            raise Fp8qError("x must be [tokens][k], got %s" % (tuple(xs),))
        if first != 0:
            raise Fp8qError("first belongs to ids")
        tokens, topk, experts = xs[0], 1, 1
        shape, stride_w, stride_s = (tokens, n), 0, 0
    if (k + 127) // 128 != kt:
        raise Fp8qError("x has K = %d, w has %d tiles of 128" % (k, kt))
    if x.is_contiguous():
        ld_x, ld_xj = (k, 0) if len(xs) == 2 else (topk * k, k)
    else:
        st = x.stride()
        if x.numel() > 0 and (st[-1] != 1 or min(st) < 0):
            raise Fp8qError("x must have a unit stride in its last dimension and no negative one")
        ld_x = k if tokens <= 1 else st[0]
        ld_xj = st[1] if len(xs) == 3 and topk > 1 else 0
    code = _out_code(out_dtype)
    ld_y = n
    if out is None:
        out = _new(shape, out_dtype, dev, stream)
    else:
        if out.dtype is not out_dtype or out.shape != shape or (out.numel() > 0 and out.stride(-1) != 1):
            raise Fp8qError("out must be %s %s with a unit stride in its last dimension, got %s %s" % (
                out_dtype, shape, out.dtype, tuple(out.shape)))
        # the rows of all routes are numbered in one go
        if routed:
            ld_y = out.stride(1) if topk > 1 else (out.stride(0) if tokens > 1 else n)
            if tokens > 1 and topk > 1 and out.stride(0) != topk * ld_y:
                raise Fp8qError("the routes of out must be equally far apart")
        elif tokens > 1:
            ld_y = out.stride(0)
        if ld_y < n and out.numel() > 0:
            raise Fp8qError("the rows of out overlap")
    lib = _library()
    if gated:
        st = _call(lib.fp4_gated_gemv_mx, dev, stream, tokens, topk, _address(ids), first, experts, n, k, x.data_ptr(),
                   ld_x, ld_xj, w.data_ptr(), ld_w, w_strides[routed], stride_w, w_scale.data_ptr(), ld_s,
                   s_strides[routed], stride_s, _act_code(act), out.data_ptr(), ld_y, code)
    else:
        st = _call(lib.fp4_gemv_mx, dev, stream, tokens, topk, _address(ids), first, experts, n, k, x.data_ptr(), ld_x,
                   ld_xj, w.data_ptr(), ld_w, stride_w, w_scale.data_ptr(), ld_s, stride_s, out.data_ptr(), ld_y, code)
    _check(st, name)
    return out


def fp4_gemv_mx(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, n: int | None = None,
                ids: torch.Tensor | None = None, first: int = 0, out_dtype=torch.bfloat16,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Few bf16 rows times an FP4 weight: ``y = x deq(w)^T``, the weight-only
    product of serving. FP32 sums, in an order that the sizes alone choose (a
    row's does not depend on what the others hold, but on their number); ``y`` in
    bf16 or FP32.

    ``x[m][k]``; ``w``, ``w_scale``: an FP4 matrix of ``n`` rows with K = ``k``
    from :func:`fp4_quantize_mx` (``n``: whole tiles of 16 when left out).
    Returns ``[m][n]``.

    With ``ids`` (int32 ``[tokens][topk]``): ``x[tokens][k]``, or
    ``[tokens][topk][k]`` where every route has a row of its own, and a stack of
    the experts' matrices ``w[E][..]``; route ``(t, j)`` goes through expert
    ``ids[t][j] - first``. Returns ``[tokens][topk][n]``, zeros for ids outside
    ``[first, first + E)`` (all of them on a rank with E = 0). Up to 4096 routes, topk up to 32.
    """
    return _gemv(x, w, w_scale, n, ids, first, False, None, out_dtype, out, stream, "fp4_gemv_mx")


def fp4_gated_gemv_mx(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, n: int | None = None,
                      act: str = "silu", ids: torch.Tensor | None = None, first: int = 0,
                      out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The first half of a gated feed-forward block for few rows:
    ``act(x Wg^T) * (x Wu^T)`` with FP4 weights, in one kernel.

    ``w[2][..]``: two stacked FP4 matrices of ``n`` rows, the gate's first (with
    ``ids``: ``w[E][2][..]``); ``act``: ``"silu"`` or ``"gelu"`` (its tanh form).
    Everything else as :func:`fp4_gemv_mx`.
    """
    return _gemv(x, w, w_scale, n, ids, first, True, act, out_dtype, out, stream, "fp4_gated_gemv_mx")
