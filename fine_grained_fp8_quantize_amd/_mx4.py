"""FP4 microscaling operators (``include/fp8q_mx4.h``): the binding of the
``fp4_*`` entry points. Imported by the package; see its docstring."""
from __future__ import annotations

import ctypes

import torch

from . import Fp8qError, _check, _check_tensor, _load, _out_code, _rowmajor

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
    return (kt, rt, 1024), ((kt + 3) // 4, rt, 64)


_WORDS = (torch.int32, torch.uint32)


def _on_gpu(*ts: torch.Tensor | None) -> int:
    """The index of the one GPU that all tensors given live on."""
    dev = None
    for t in ts:
        if t is None:
            continue
        d = t.get_device()
        if d != dev:
            if d < 0:
                raise Fp8qError("fp8q tensors must live on the GPU (got a %s tensor)" % t.device)
            if dev is not None:
                raise Fp8qError("all tensors must be on one device (got cuda:%d and cuda:%d)" % (dev, d))
            dev = d
    return dev


def _address(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.data_ptr()


def _raw_stream(stream, dev: int) -> int:
    """hipStream_t of ``stream``, or of torch's current stream on ``dev``. (A
    call with few rows takes the GPU a few microseconds, and making a Stream
    object takes the host as long.)"""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(dev)


def _call(fn, dev: int, stream, *args) -> int:
    """Status of the C call ``fn`` for tensors of GPU ``dev``. The call launches on
    the current device when the stream is the default one, whose handle is the
    same on every GPU."""
    if dev == torch._C._cuda_getDevice():
        return fn(*args, _raw_stream(stream, dev))
    with torch.cuda.device(dev):
        return fn(*args, _raw_stream(stream, dev))


def _new(shape, dtype, dev: int, stream) -> torch.Tensor:
    """A new tensor, its memory taken on ``stream`` (see ``_empty``)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=_device(dev))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=_device(dev))


_devices: dict = {}


def _device(dev: int) -> torch.device:
    got = _devices.get(dev)
    if got is None:
        got = _devices[dev] = torch.device("cuda", dev)
    return got


def _tiles_ld(t: torch.Tensor, unit: int, lead: int, what: str) -> int:
    """Row tiles between two K tiles (or K groups) of ``t``, whose row tiles of
    ``unit`` elements must be contiguous."""
    shape = t.shape
    rt = shape[-2]
    if t.is_contiguous() or t.numel() == 0:
        return rt
    st = t.stride()
    if st[-1] != 1 or (rt > 1 and st[-2] != unit):
        raise Fp8qError("the row tiles of %s must be contiguous" % what)
    if min(st) < 0 or st[-3] % unit != 0:
        raise Fp8qError("%s must have K tiles a whole number of row tiles apart" % what)
    return rt if shape[-3] <= 1 else st[-3] // unit


def _matrix(q: torch.Tensor, scale: torch.Tensor, what: str, lead: int = 0):
    """Checks the two tensors of an FP4 matrix (or of a stack of them, with
    ``lead`` = 1) against each other: dtypes, shapes, tiles contiguous. Returns
    K tiles, row tiles, and the leading dimensions of codes and scales."""
    qs, ss = q.shape, scale.shape
    if (lead == 0 and q.dtype is torch.uint8 and scale.dtype is torch.int32 and q.is_contiguous()
            and scale.is_contiguous() and len(qs) == 3 and qs[2] == 1024):
        kt, rt, _ = qs  # the usual case, in few steps
        if ss == ((kt + 3) // 4, rt, 64):
            return kt, rt, rt, rt
    if q.dtype is not torch.uint8 or len(qs) != 3 + lead or qs[-1] != 1024:
        raise Fp8qError("%s must be uint8 %s[k tiles][row tiles][1024]" % (what, "[E]" * lead))
    kt, rt = qs[-3], qs[-2]
    if (scale.dtype not in _WORDS or len(ss) != 3 + lead or ss[-1] != 64 or ss[-2] != rt or ss[-3] != (kt + 3) // 4
            or (lead and ss[0] != qs[0])):
        raise Fp8qError("%s_scale must be int32 %s, got %s %s" % (
            what, (*qs[:lead], (kt + 3) // 4, rt, 64), scale.dtype, tuple(ss)))
    return kt, rt, _tiles_ld(q, 1024, lead, what), _tiles_ld(scale, 64, lead, what + "_scale")


def _output(out, shape, dtype, dev, stream) -> torch.Tensor:
    """The output: new when absent, otherwise of exactly this dtype and shape
    with unit column stride."""
    if out is None:
        return _new(shape, dtype, dev, stream)
    _check_tensor(out, shape, (dtype,), "out")
    return out


def _codes_out(q, scale, q_shape, s_shape, dev, stream, lead: int = 0):
    """Code and scale outputs: new when absent, checked otherwise; with their
    leading dimensions."""
    if q is None:
        q = _new(q_shape, torch.uint8, dev, stream)
    if scale is None:
        scale = _new(s_shape, torch.int32, dev, stream)
    if q.shape != q_shape or scale.shape != s_shape:
        raise Fp8qError("q and scale have shapes %s and %s, expected %s and %s" % (
            tuple(q.shape), tuple(scale.shape), q_shape, s_shape))
    return (q, scale, *_matrix(q, scale, "q", lead)[2:])


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
    dev = _on_gpu(x, q, scale)
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
    q, scale, ld_q, ld_s = _codes_out(q, scale, q_shape, s_shape, dev, stream, lead)
    groups = x.shape[0] if lead else 1
    ld_x = cols if rows <= 1 else x.stride(-2)
    st = _call(_library().fp4_quantize_mx, dev, stream, groups, x.data_ptr(), rows, cols, ld_x,
               x.stride(0) if lead else 0, t, q.data_ptr(), ld_q, q.stride(0) if lead else 0, scale.data_ptr(), ld_s,
               scale.stride(0) if lead else 0)
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
    dev = _on_gpu(x, dst_rows, q, scale)
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
    q, scale, ld_q, ld_s = _codes_out(q, scale, *_shapes(m_total, cols), dev, stream)
    ld_x = cols if tokens <= 1 else x.stride(0)
    st = _call(_library().fp4_quantize_mx_scatter, dev, stream, x.data_ptr(), tokens, cols, ld_x, dst_rows.shape[1],
               dst_rows.data_ptr(), m_total, q.data_ptr(), ld_q, scale.data_ptr(), ld_s)
    _check(st, "fp4_quantize_mx_scatter")
    return q, scale


def fp4_dequantize_mx(q: torch.Tensor, scale: torch.Tensor, rows: int, cols: int, out_dtype=torch.bfloat16,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values ``[rows][cols]`` (bf16 or fp32, exact in both) that an FP4
    matrix of ``rows`` rows with K = ``cols`` holds."""
    dev = _on_gpu(q, scale, out)
    kt, rt, ld_q, ld_s = _matrix(q, scale, "q")
    if (kt, rt) != _shapes(rows, cols)[0][:2]:
        raise Fp8qError("q has %d x %d tiles, which is not a matrix of %d rows with K = %d" % (kt, rt, rows, cols))
    oc = _out_code(out_dtype)
    out = _output(out, (rows, cols), out_dtype, dev, stream)
    st = _call(_library().fp4_dequantize_mx, dev, stream, q.data_ptr(), ld_q, scale.data_ptr(), ld_s, rows, cols,
               out.data_ptr(), cols if rows <= 1 else out.stride(0), oc)
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
    dev = _on_gpu(a, a_scale, b, b_scale, out)
    kt, rta, ld_a, ld_as = _matrix(a, a_scale, "a")
    ktb, rtb, ld_b, ld_bs = _matrix(b, b_scale, "b")
    if kt != ktb:
        raise Fp8qError("a and b disagree on K (%d vs %d tiles of 128)" % (kt, ktb))
    m, n = _rows_of(m, rta, "m"), _rows_of(n, rtb, "n")
    oc = _out_code(out_dtype)
    out = _output(out, (m, n), out_dtype, dev, stream)
    st = _call(_library().fp4_gemm_mx, dev, stream, m, n, kt * 128, a.data_ptr(), ld_a, a_scale.data_ptr(), ld_as,
               b.data_ptr(), ld_b, b_scale.data_ptr(), ld_bs, out.data_ptr(), n if m <= 1 else out.stride(0), oc)
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
    dev = _on_gpu(a, a_scale, b, b_scale, group_offsets, group_rows, out)
    kt, rta, ld_a, ld_as = _matrix(a, a_scale, "a")
    ktb, rtb, ld_b, ld_bs = _matrix(b, b_scale, "b", 1)
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
    out = _output(out, (m_total, n), out_dtype, dev, stream)
    if groups == 0:  # (the C call has nothing to do then)
        with torch.cuda.stream(stream or torch.cuda.current_stream(dev)):
            return out.zero_()
    st = _call(_library().fp4_grouped_gemm_mx, dev, stream, groups, group_offsets.data_ptr(), _address(group_rows),
               m_total, n, kt * 128, a.data_ptr(), ld_a, a_scale.data_ptr(), ld_as, b.data_ptr(), ld_b, b.stride(0),
               b_scale.data_ptr(), ld_bs, b_scale.stride(0), out.data_ptr(), n if m_total <= 1 else out.stride(0), oc)
    _check(st, "fp4_grouped_gemm_mx")
    return out
