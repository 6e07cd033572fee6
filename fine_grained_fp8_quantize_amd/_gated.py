"""Gated feed-forward operators (``include/fp8q_gated.h``): the binding of
``fp8_gated_gemm``, ``fp8_grouped_gated_gemm`` and ``fp8_gated_backward``.
Imported by the package; see its docstring."""
from __future__ import annotations

import ctypes

import torch

from . import OUT_BF16, OUT_F32, Fp8qError, _check, _check_tensor, _codes, _load, _rowmajor
from ._mx4 import _address, _call, _new, _on_gpu

ACT_SILU = 0
ACT_GELU = 1
OUT_E4M3 = 2

_ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU}
_OUTS = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32, torch.float8_e4m3fn: OUT_E4M3}
_CODES = (torch.float8_e4m3fn, torch.uint8)

_lib = None


def _library():
    """The C library with the signatures of the gated entry points."""
    global _lib
    if _lib is None:
        L = _load()
        p, i64, i32, cint = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
        L.fp8_gated_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8_gated_workspace_bytes.restype = i64
        L.fp8_gated_gemm.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, i64, p, i64, i64, cint, p, i64, cint, p,
                                     i64, p, i64, p, i64, p]
        L.fp8_grouped_gated_gemm.argtypes = [i32, p, p, i64, i64, i64, p, i64, p, i64, p, i64, i64, i64, p, i64, i64,
                                             i64, cint, p, i64, cint, p, i64, p, i64, p, i64, p]
        L.fp8_grouped_gated_workspace_bytes.argtypes = [i64, i64]
        L.fp8_grouped_gated_workspace_bytes.restype = i64
        L.fp8_gated_backward.argtypes = [i64, i64, p, i64, p, i64, cint, cint, p, i64, p, i64, p, i64, p, i64, p]
        for name in ("fp8_gated_gemm", "fp8_grouped_gated_gemm", "fp8_gated_backward"):
            getattr(L, name).restype = cint
        _lib = L
    return _lib


def _act_code(act: str) -> int:
    code = _ACTS.get(act)
    if code is None:
        raise Fp8qError("act must be 'silu' or 'gelu'")
    return code


def _out_code(dtype, allowed) -> int:
    if dtype not in allowed:
        raise Fp8qError("out_dtype must be one of %s" % ", ".join(str(d) for d in allowed))
    return _OUTS[dtype]


_GRADS = (torch.float8_e4m3fn, torch.bfloat16)


def _ld(t: torch.Tensor) -> int:
    """Leading dimension of a row-major matrix (a lone row has none)."""
    return t.shape[1] if t.shape[0] <= 1 else t.stride(0)


def _matrix_out(t, shape, dtypes, dev, stream, what: str) -> torch.Tensor:
    """An output matrix: new when absent, checked otherwise."""
    if t is None:
        return _new(shape, dtypes[0], dev, stream)
    if dtypes[0] is torch.float32:
        _f32(t, shape, what)
    else:
        _check_tensor(t, shape, dtypes, what)
    return t


def _f32(t: torch.Tensor, shape, what: str) -> None:
    """An FP32 matrix of scales; the stride along one row of one column does not matter."""
    if t.dim() > 0 and t.shape[-1] == 1:
        t = t.as_strided(t.shape, (*t.stride()[:-1], 1))
    _check_tensor(t, shape, (torch.float32,), what)


def _operands(a, a_scale, b, b_scale, lead: int):
    """Checked A and W of the gated products; m, n, k, the leading dimensions of A and its scales, and the weights'
    strides."""
    if a.dim() == 2:
        m, k = a.shape
        bs, ss = b.shape, b_scale.shape
        n = bs[-2] if len(bs) > 2 else -1
        f32 = torch.float32
        if (a.dtype in _CODES and b.dtype in _CODES and a_scale.dtype is f32 and b_scale.dtype is f32
                and bs[lead:] == (2, n, k) and len(bs) == 3 + lead and k % 128 == 0 and a.is_contiguous()
                and b.is_contiguous() and a_scale.is_contiguous() and b_scale.is_contiguous()
                and a_scale.shape == (k // 128, m) and ss[lead:] == (2, -(-n // 128), k // 128)
                and ss[:lead] == bs[:lead]):
            return m, n, k, k, m, (k, n * k), (k // 128, ss[-2] * ss[-1])  # the usual case, in few steps
    _rowmajor(_codes(a, "a"), "a")
    _codes(b, "b")
    what = "[E][2][n][k]" if lead else "[2][n][k]"
    if b.dim() != 3 + lead or b.shape[lead] != 2:
        raise Fp8qError("b must be %s codes, gate first" % what)
    m, k = a.shape
    n, kb = b.shape[-2:]
    if kb != k:
        raise Fp8qError("a and b disagree on K (%d vs %d)" % (k, kb))
    if k % 128:
        raise Fp8qError("K must be a multiple of 128, got %d" % k)
    if b.numel() > 0 and (b.stride(-1) != 1 or min(b.stride()) < 0):
        raise Fp8qError("b must have a unit column stride and no negative one")
    _f32(a_scale, (k // 128, m), "a_scale")
    _f32(b_scale, (*b.shape[:-2], -(-n // 128), k // 128), "b_scale")
    ldb = k if n <= 1 else b.stride(-2)
    ld_bs = k // 128 if b_scale.shape[-2] <= 1 else b_scale.stride(-2)
    return m, n, k, _ld(a), _ld(a_scale), (ldb, b.stride(lead)), (ld_bs, b_scale.stride(lead))


def _outputs(m, n, out_dtype, out, scale, gate_up, dev, stream):
    """H, its scales (E4M3) and gate_up: new when absent (gate_up: not kept), checked otherwise. With the arguments of
    the C call."""
    code = _out_code(out_dtype, _OUTS)
    ld_o = n
    if code == OUT_E4M3:
        if n % 128:
            raise Fp8qError("E4M3 output needs n in whole 1x128 tiles, got %d" % n)
        if out is None:
            out = _new((m, n), torch.float8_e4m3fn, dev, stream)
        else:
            _check_tensor(out, (m, n), _CODES, "out")
            ld_o = _ld(out)
        if scale is None:
            scale, ld_s = _new((n // 128, m), torch.float32, dev, stream), m
        else:
            _f32(scale, (n // 128, m), "scale")
            ld_s = _ld(scale)
    else:
        if scale is not None:
            raise Fp8qError("scale belongs to E4M3 output")
        ld_s = 0
        if out is None:
            out = _new((m, n), out_dtype, dev, stream)
        else:
            _check_tensor(out, (m, n), (out_dtype,), "out")
            ld_o = _ld(out)
    ld_g = 0
    if gate_up is not None:
        ld_g = 2 * n
        if gate_up.dtype is not torch.bfloat16 or gate_up.shape != (m, ld_g) or not gate_up.is_contiguous():
            _check_tensor(gate_up, (m, ld_g), (torch.bfloat16,), "gate_up")
            ld_g = _ld(gate_up)
    tail = (out.data_ptr(), ld_o, code, _address(scale), ld_s, _address(gate_up), ld_g)
    return out, scale, tail


def _scratch(workspace, need: int, dev, stream):
    """A workspace: new when absent (None if none is needed), checked otherwise."""
    if workspace is None:
        return _new(need, torch.uint8, dev, stream) if need else None
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise Fp8qError("workspace must be a contiguous uint8 tensor")
    return workspace


def fp8_gated_gemm(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, act: str = "silu",
                   out_dtype=torch.bfloat16, out: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                   gate_up: torch.Tensor | None = None, stream=None, workspace: torch.Tensor | None = None):
    """The first half of a gated feed-forward block in one kernel:
    ``H = act(A Wg^T) * (A Wu^T)``.

    ``a[m][k]`` E4M3 codes with ``a_scale[k/128][m]`` (:func:`fp8_quantize_act`);
    ``b[2][n][k]`` codes, the gate's first, with ``b_scale[2][ceil(n/128)][k/128]``
    (:func:`fp8_quantize_weight_grouped` of two matrices, or a ``[2n][k]``
    :func:`fp8_quantize_weight` seen as that, where n is a multiple of 128).
    ``act``: ``"silu"`` or ``"gelu"`` (its tanh form).

    Returns ``H[m][n]`` in bf16 or FP32, or, with ``out_dtype =
    torch.float8_e4m3fn``, its codes and scales ``[n/128][m]`` in 1x128 tiles:
    the operand of the down product. ``gate_up``: a bf16 ``[m][2n]`` tensor that
    takes the two products, for :func:`fp8_gated_backward`. ``workspace``: uint8
    scratch for E4M3 output of few rows (taken from torch when left out).
    """
    dev = _on_gpu(a, a_scale, b, b_scale, out, scale, gate_up, workspace)
    m, n, k, lda, ld_as, (ldb, stride_b), (ld_bs, stride_bs) = _operands(a, a_scale, b, b_scale, 0)
    code = _act_code(act)
    out, scale, tail = _outputs(m, n, out_dtype, out, scale, gate_up, dev, stream)
    lib = _library()
    if workspace is not None or scale is not None:
        workspace = _scratch(workspace, lib.fp8_gated_workspace_bytes(m, n, k), dev, stream)
    st = _call(lib.fp8_gated_gemm, dev, stream, m, n, k, a.data_ptr(), lda, a_scale.data_ptr(), ld_as,
               b.data_ptr(), ldb, stride_b, b_scale.data_ptr(), ld_bs, stride_bs, code, *tail, _address(workspace),
               0 if workspace is None else workspace.numel())
    _check(st, "fp8_gated_gemm")
    return out if scale is None else (out, scale)


def fp8_grouped_gated_gemm(group_offsets: torch.Tensor, group_rows: torch.Tensor | None, a: torch.Tensor,
                           a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor, act: str = "silu",
                           out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                           scale: torch.Tensor | None = None, gate_up: torch.Tensor | None = None, stream=None,
                           workspace: torch.Tensor | None = None):
    """:func:`fp8_gated_gemm` for the experts of an expert-sorted row layout
    (:func:`moe_dispatch` with ``align=128``): rows ``[off[e], off[e+1])`` of ``a``
    with ``b[e]``, of which the first ``group_rows[e]`` are real (None: all,
    which may take the sums in another order than counts that say the same).

    ``group_offsets`` int32 ``[E+1]``, multiples of 128, its last entry
    ``m_total``, the rows of ``a``; ``b[E][2][n][k]`` with
    ``b_scale[E][2][ceil(n/128)][k/128]``. Padding rows of all outputs are zeros.
    ``workspace`` is that of E4M3 output, as there.
    """
    dev = _on_gpu(a, a_scale, b, b_scale, group_offsets, group_rows, out, scale, gate_up, workspace)
    m, n, k, lda, ld_as, (ldb, stride_b), (ld_bs, stride_bs) = _operands(a, a_scale, b, b_scale, 1)
    groups = b.shape[0]
    for t, entries, name in ((group_offsets, groups + 1, "group_offsets"), (group_rows, groups, "group_rows")):
        if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or t.numel() != entries or not t.is_contiguous()):
            raise Fp8qError("%s must be a contiguous int32 tensor of %d entries" % (name, entries))
    code = _act_code(act)
    if groups == 0 and m > 0:
        raise Fp8qError("%d rows belong to no expert" % m)
    out, scale, tail = _outputs(m, n, out_dtype, out, scale, gate_up, dev, stream)
    lib = _library()
    if workspace is not None or scale is not None:
        workspace = _scratch(workspace, lib.fp8_grouped_gated_workspace_bytes(m, n), dev, stream)
    st = _call(lib.fp8_grouped_gated_gemm, dev, stream, groups, group_offsets.data_ptr(), _address(group_rows),
               m, n, k, a.data_ptr(), lda, a_scale.data_ptr(), ld_as, b.data_ptr(), ldb, stride_b,
               b.stride(0), b_scale.data_ptr(), ld_bs, stride_bs, b_scale.stride(0), code, *tail, _address(workspace),
               0 if workspace is None else workspace.numel())
    _check(st, "fp8_grouped_gated_gemm")
    return out if scale is None else (out, scale)


def fp8_gated_backward(dh: torch.Tensor, gate_up: torch.Tensor, act: str = "silu", out_dtype=torch.float8_e4m3fn,
                       transposed: bool = False, out: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                       out_t: torch.Tensor | None = None, scale_t: torch.Tensor | None = None, stream=None):
    """The gradients of gate and up, side by side as ``D[m][2n]`` (the gate's
    first), from bf16 ``dh[m][n]``, the gradient of H, and the ``gate_up[m][2n]``
    that :func:`fp8_gated_gemm` kept: ``dG = dH U act'(G)``, ``dU = dH act(G)``.

    ``out_dtype=torch.float8_e4m3fn``: returns codes ``[m][2n]`` and scales
    ``[2n/128][m]`` in 1x128 tiles (for the product with the transposed weights,
    dX) and, with ``transposed``, codes ``[2n][m]`` and scales ``[m/128][2n]`` in
    128x1 token tiles too (for the product with X, dW; m a multiple of 128). A
    tile that holds a NaN or an infinity reads back with nothing finite in it.
    ``torch.bfloat16``: returns D in bf16, any n.
    """
    dev = _on_gpu(dh, gate_up, out, scale, out_t, scale_t)
    code = _out_code(out_dtype, _GRADS)
    if dh.dtype is not torch.bfloat16:
        raise Fp8qError("dh must be bfloat16")
    if dh.dim() != 2:
        raise Fp8qError("dh must be [m][n]")
    m, n = dh.shape
    if gate_up.dtype is torch.bfloat16 and gate_up.shape == (m, 2 * n) and dh.is_contiguous() and gate_up.is_contiguous():
        ld_dh, ld_g = n, 2 * n
    else:
        _check_tensor(dh, (m, n), (torch.bfloat16,), "dh")
        _check_tensor(gate_up, (m, 2 * n), (torch.bfloat16,), "gate_up")
        ld_dh, ld_g = _ld(dh), _ld(gate_up)
    given = out is not None or scale is not None or out_t is not None or scale_t is not None
    if code == OUT_BF16:
        if transposed or scale is not None or out_t is not None or scale_t is not None:
            raise Fp8qError("scales and transposed codes belong to E4M3 output")
        out = _matrix_out(out, (m, 2 * n), (torch.bfloat16,), dev, stream, "out")
    else:
        if n % 128:
            raise Fp8qError("E4M3 output needs n in whole 1x128 tiles, got %d" % n)
        if transposed and m % 128:
            raise Fp8qError("transposed codes need m in whole 128x1 tiles, got %d" % m)
        if not transposed and (out_t is not None or scale_t is not None):
            raise Fp8qError("out_t and scale_t belong to transposed=True")
        out = _matrix_out(out, (m, 2 * n), _CODES, dev, stream, "out")
        scale = _matrix_out(scale, (n // 64, m), (torch.float32,), dev, stream, "scale")
        if transposed:
            out_t = _matrix_out(out_t, (2 * n, m), _CODES, dev, stream, "out_t")
            scale_t = _matrix_out(scale_t, (m // 128, 2 * n), (torch.float32,), dev, stream, "scale_t")
    lds = [0 if t is None else _ld(t) for t in (out, scale, out_t, scale_t)] if given else (2 * n, m, m, 2 * n)
    st = _call(_library().fp8_gated_backward, dev, stream, m, n, dh.data_ptr(), ld_dh, gate_up.data_ptr(), ld_g,
               _act_code(act), code, out.data_ptr(), lds[0], _address(scale), lds[1], _address(out_t), lds[2],
               _address(scale_t), lds[3])
    _check(st, "fp8_gated_backward")
    if code == OUT_BF16:
        return out
    return (out, scale, out_t, scale_t) if transposed else (out, scale)
