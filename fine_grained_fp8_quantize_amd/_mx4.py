"""FP4 microscaling operators (``include/fp8q_mx4.h``): the binding of the
``fp4_*`` entry points. Imported by the package; see its docstring."""
from __future__ import annotations

import ctypes

import torch

from . import (Fp8qError, _check, _check_tensor, _empty, _load, _need_gpu, _out_code, _ptr, _rowmajor, _stream)

FP4_TILE_1x32 = 0
FP4_TILE_32x1 = 1

_lib = None


def _library():
    """The C library with the signatures of the FP4 entry points."""
    global _lib
    if _lib is None:
        L = _load()
        p, i64, i32, cint = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
        L.fp4_quantize_mx.argtypes = [i32, p, i64, i64, i64, i64, cint, p, i64, i64, p, i64, i64, p]
        L.fp4_quantize_mx_scatter.argtypes = [p, i64, i64, i64, i32, p, i64, p, i64, p, i64, p]
        L.fp4_dequantize_mx.argtypes = [p, i64, p, i64, i64, i64, p, i64, cint, p]
        L.fp4_gemm_mx.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p, i64, cint, p]
        L.fp4_grouped_gemm_mx.argtypes = [i32, p, p, i64, i64, i64, p, i64, p, i64, p, i64, i64, p, i64, i64,
                                          p, i64, cint, p]
        for name in ("fp4_quantize_mx", "fp4_quantize_mx_scatter", "fp4_dequantize_mx", "fp4_gemm_mx",
                     "fp4_grouped_gemm_mx"):
            getattr(L, name).restype = cint
        _lib = L
    return _lib


def _shapes(rows: int, k: int):
    """Shapes of the code and scale tensors of an FP4 matrix [rows][k]."""
    kt, rt = -(-k // 128), -(-rows // 16)
    return (kt, rt, 1024), (-(-kt // 4), rt, 64)


def _matrix(q: torch.Tensor, scale: torch.Tensor, what: str, lead: int = 0):
    """Checks the two tensors of an FP4 matrix (or of a stack of them, with
    ``lead`` = 1) against each other: dtypes, shapes, tiles contiguous.
    Returns (K tiles, row tiles)."""
    if q.dtype != torch.uint8 or q.dim() != 3 + lead or q.shape[-1] != 1024:
        raise Fp8qError("%s must be uint8 %s[k tiles][row tiles][1024]" % (what, "[E]" * lead))
    kt, rt = q.shape[-3], q.shape[-2]
    want = (*q.shape[:lead], -(-kt // 4), rt, 64)
    if scale.dtype not in (torch.int32, torch.uint32) or tuple(scale.shape) != want:
        raise Fp8qError("%s_scale must be int32 %s, got %s %s" % (what, want, scale.dtype, tuple(scale.shape)))
    for t, unit in ((q, 1024), (scale, 64)):
        if t.numel() and (t.stride(-1) != 1 or (rt > 1 and t.stride(-2) != unit)):
            raise Fp8qError("the row tiles of %s must be contiguous" % what)
        if t.numel() and (t.stride(-3) < 0 or t.stride(-3) % unit != 0 or any(t.stride(i) < 0 for i in range(lead))):
            raise Fp8qError("%s must have K tiles a whole number of row tiles apart" % what)
    return kt, rt


def _ld(t: torch.Tensor, unit: int) -> int:
    """Row tiles between two K tiles (or K groups) of a checked tensor."""
    return t.shape[-2] if t.shape[-3] <= 1 else t.stride(-3) // unit


def _same_device(*ts: torch.Tensor) -> None:
    for t in ts:
        if t is not None and t.device != ts[0].device:
            raise Fp8qError("all tensors must be on one device (got %s and %s)" % (ts[0].device, t.device))


def fp4_quantize_mx(x: torch.Tensor, tiling: str = "1x32", q: torch.Tensor | None = None,
                    scale: torch.Tensor | None = None, stream=None):
    """Microscaling quantization to FP4 (E2M1 codes, one power-of-two scale
    per 32 elements), in the tile layout that the FP4 products read.

    ``x``: bf16 ``[rows][cols]``, or ``[E][rows][cols]`` for a stack (say the
    experts' weights) in one launch; unit column stride, any row stride.
    ``tiling="1x32"``: blocks along each row, an FP4 matrix of ``rows`` rows
    with K = ``cols``. ``tiling="32x1"``: blocks down each column, the
    transposed operand: ``cols`` rows with K = ``rows``.
    Returns ``q`` uint8 ``[k tiles][row tiles][1024]`` and ``scale`` int32
    ``[ceil(k tiles / 4)][row tiles][64]`` (with ``[E]`` in front for a
    stack), K tiles of 128 and row tiles of 16.
    """
    _need_gpu(x, q, scale)
    _same_device(x, q, scale)
    if x.dtype != torch.bfloat16:
        raise Fp8qError("x must be bfloat16")
    lead = x.dim() - 2
    if lead not in (0, 1) or (x.numel() > 0 and x.stride(-1) != 1):
        raise Fp8qError("x must be [rows][cols] or [E][rows][cols] with unit column stride")
    if x.numel() > 0 and any(x.stride(i) < 0 for i in range(x.dim())):
        raise Fp8qError("x has a negative stride")
    t = {"1x32": FP4_TILE_1x32, "32x1": FP4_TILE_32x1}.get(tiling)
    if t is None:
        raise Fp8qError("tiling must be '1x32' or '32x1'")
    rows, cols = x.shape[-2:]
    out_rows, k = (rows, cols) if t == FP4_TILE_1x32 else (cols, rows)
    q_shape, s_shape = (tuple(x.shape[:lead]) + s for s in _shapes(out_rows, k))
    if q is None:
        q = _empty(q_shape, torch.uint8, x.device, stream)
    if scale is None:
        scale = _empty(s_shape, torch.int32, x.device, stream)
    _check_tensor(q, q_shape, (torch.uint8,), "q")
    _check_tensor(scale, s_shape, (torch.int32, torch.uint32), "scale")
    _matrix(q, scale, "q", lead)
    groups = x.shape[0] if lead else 1
    ld_x = cols if rows <= 1 else x.stride(-2)
    st = _library().fp4_quantize_mx(
        groups, _ptr(x), rows, cols, ld_x, x.stride(0) if lead else 0, t,
        _ptr(q), _ld(q, 1024), q.stride(0) if lead else 0,
        _ptr(scale), _ld(scale, 64), scale.stride(0) if lead else 0, _stream(stream))
    _check(st, "fp4_quantize_mx")
    return q, scale


def fp4_quantize_mx_scatter(x: torch.Tensor, dst_rows: torch.Tensor, m_total: int, q: torch.Tensor | None = None,
                            scale: torch.Tensor | None = None, stream=None):
    """Quantize bf16 token rows ``x[tokens][cols]`` to FP4 once and store each
    to its expert-sorted destination rows (``dst_rows`` int32
    ``[tokens][topk]``, topk 1..8, -1 for no route; see :func:`moe_dispatch`).

    Returns the FP4 matrix ``(q, scale)`` of ``m_total`` rows with K =
    ``cols``; rows no route names (segment padding) are left as they were.
    """
    _need_gpu(x, dst_rows, q, scale)
    _same_device(x, dst_rows, q, scale)
    _rowmajor(x, "x")
    if x.dtype != torch.bfloat16:
        raise Fp8qError("x must be bfloat16")
    if x.numel() > 0 and x.stride(0) < 0:
        raise Fp8qError("x has a negative stride")
    tokens, cols = x.shape
    if dst_rows.dtype != torch.int32 or dst_rows.dim() != 2 or dst_rows.shape[0] != tokens:
        raise Fp8qError("dst_rows must be int32 [tokens][topk]")
    if not dst_rows.is_contiguous():
        raise Fp8qError("dst_rows must be contiguous [tokens][topk]")
    q_shape, s_shape = _shapes(m_total, cols)
    if q is None:
        q = _empty(q_shape, torch.uint8, x.device, stream)
    if scale is None:
        scale = _empty(s_shape, torch.int32, x.device, stream)
    _check_tensor(q, q_shape, (torch.uint8,), "q")
    _check_tensor(scale, s_shape, (torch.int32, torch.uint32), "scale")
    _matrix(q, scale, "q")
    ld_x = cols if tokens <= 1 else x.stride(0)
    st = _library().fp4_quantize_mx_scatter(_ptr(x), tokens, cols, ld_x, dst_rows.shape[1], _ptr(dst_rows), m_total,
                                            _ptr(q), _ld(q, 1024), _ptr(scale), _ld(scale, 64), _stream(stream))
    _check(st, "fp4_quantize_mx_scatter")
    return q, scale


def fp4_dequantize_mx(q: torch.Tensor, scale: torch.Tensor, rows: int, cols: int, out_dtype=torch.bfloat16,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values ``[rows][cols]`` (bf16 or fp32, exact in both) that an FP4
    matrix of ``rows`` rows with K = ``cols`` holds."""
    _need_gpu(q, scale, out)
    _same_device(q, scale, out)
    kt, rt = _matrix(q, scale, "q")
    if (kt, rt) != _shapes(rows, cols)[0][:2]:
        raise Fp8qError("q has %d x %d tiles, which is not a matrix of %d rows with K = %d" % (kt, rt, rows, cols))
    oc = _out_code(out_dtype)
    if out is None:
        out = _empty((rows, cols), out_dtype, q.device, stream)
    _check_tensor(out, (rows, cols), (out_dtype,), "out")
    st = _library().fp4_dequantize_mx(_ptr(q), _ld(q, 1024), _ptr(scale), _ld(scale, 64), rows, cols, _ptr(out),
                                      cols if rows <= 1 else out.stride(0), oc, _stream(stream))
    _check(st, "fp4_dequantize_mx")
    return out


def _rows_of(rows, tiles: int, what: str) -> int:
    """The logical row count of an FP4 matrix: whole tiles unless given."""
    if rows is None:
        return tiles * 16
    if -(-int(rows) // 16) != tiles:
        raise Fp8qError("%s = %d does not fit %d row tiles of 16" % (what, rows, tiles))
    return int(rows)


def fp4_gemm_mx(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                m: int | None = None, n: int | None = None, out_dtype=torch.bfloat16,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``C[m][n] = sum_k deq(A)[m][k] deq(B)[n][k]`` of two FP4 matrices from
    :func:`fp4_quantize_mx` (either tiling): a layer's forward product, and
    both gradients with the transposed operands. ``m`` and ``n`` are the
    operands' row counts (whole tiles of 16 when left out)."""
    _need_gpu(a, a_scale, b, b_scale, out)
    _same_device(a, a_scale, b, b_scale, out)
    kt, rta = _matrix(a, a_scale, "a")
    ktb, rtb = _matrix(b, b_scale, "b")
    if kt != ktb:
        raise Fp8qError("a and b disagree on K (%d vs %d tiles of 128)" % (kt, ktb))
    m, n = _rows_of(m, rta, "m"), _rows_of(n, rtb, "n")
    oc = _out_code(out_dtype)
    if out is None:
        out = _empty((m, n), out_dtype, a.device, stream)
    _check_tensor(out, (m, n), (out_dtype,), "out")
    st = _library().fp4_gemm_mx(m, n, kt * 128, _ptr(a), _ld(a, 1024), _ptr(a_scale), _ld(a_scale, 64),
                                _ptr(b), _ld(b, 1024), _ptr(b_scale), _ld(b_scale, 64),
                                _ptr(out), n if m <= 1 else out.stride(0), oc, _stream(stream))
    _check(st, "fp4_gemm_mx")
    return out


def fp4_grouped_gemm_mx(group_offsets: torch.Tensor, group_rows: torch.Tensor | None, a: torch.Tensor,
                        a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, n: int | None = None,
                        out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The experts' FP4 products: rows ``[off[e], off[e+1])`` of ``a`` times
    ``b[e]``, of which the first ``group_rows[e]`` are real.

    ``group_offsets`` int32 ``[E+1]``, multiples of 16; ``group_rows`` int32
    ``[E]`` or None. ``a`` is an FP4 matrix of ``m_total`` rows (its row tiles
    times 16), which may be more than ``group_offsets[E]``; ``b[E][..]`` the
    stacked FP4 weights of ``n`` rows each. Returns ``out[m_total][n]`` with
    padding rows, and rows past the last segment, zero.
    """
    _need_gpu(group_offsets, group_rows, a, a_scale, b, b_scale, out)
    _same_device(a, a_scale, b, b_scale, out, group_offsets, group_rows)
    kt, rta = _matrix(a, a_scale, "a")
    ktb, rtb = _matrix(b, b_scale, "b", 1)
    if kt != ktb:
        raise Fp8qError("a and b disagree on K (%d vs %d tiles of 128)" % (kt, ktb))
    groups = b.shape[0]
    if group_offsets.dtype != torch.int32 or (group_rows is not None and group_rows.dtype != torch.int32):
        raise Fp8qError("group_offsets / group_rows must be int32")
    if group_offsets.dim() != 1 or group_offsets.numel() != groups + 1 or not group_offsets.is_contiguous():
        raise Fp8qError("group_offsets needs E+1 contiguous entries")
    if group_rows is not None and (group_rows.dim() != 1 or group_rows.numel() != groups
                                   or not group_rows.is_contiguous()):
        raise Fp8qError("group_rows needs E contiguous entries")
    m_total, n = rta * 16, _rows_of(n, rtb, "n")
    oc = _out_code(out_dtype)
    if out is None:
        out = _empty((m_total, n), out_dtype, a.device, stream)
    _check_tensor(out, (m_total, n), (out_dtype,), "out")
    st = _library().fp4_grouped_gemm_mx(
        groups, _ptr(group_offsets), _ptr(group_rows), m_total, n, kt * 128, _ptr(a), _ld(a, 1024), _ptr(a_scale),
        _ld(a_scale, 64), _ptr(b), _ld(b, 1024), b.stride(0), _ptr(b_scale), _ld(b_scale, 64), b_scale.stride(0),
        _ptr(out), n if m_total <= 1 else out.stride(0), oc, _stream(stream))
    _check(st, "fp4_grouped_gemm_mx")
    return out
