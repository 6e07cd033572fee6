"""MoE routing operators (``include/fp8q_moe.h``): the binding of the
``moe_*`` entry points. Imported by the package; see its docstring."""
from __future__ import annotations

import ctypes

import torch

from . import Fp8qError, _check, _check_tensor, _load
from ._mx4 import _address, _call, _new, _on_gpu

SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
LOGITS_BF16 = 0
LOGITS_F32 = 1
MOE_MAX_EXPERTS = 1024
MOE_MAX_TOPK = 8
# device bytes moe_dispatch needs (FP8Q_MOE_DISPATCH_WORKSPACE_BYTES)
MOE_DISPATCH_WORKSPACE_BYTES = 64 * 1024 * 4

_lib = None


def _library():
    """The C library with the signatures of the MoE entry points."""
    global _lib
    if _lib is None:
        L = _load()
        p, i64, i32, cint, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float
        L.moe_dispatch.argtypes = [p, i64, i32, i32, i32, i32, p, p, p, p, i64, p]
        L.moe_balance_workspace_bytes.argtypes = [i64, i32, i64]
        L.moe_balance_loss.argtypes = [p, cint, i64, i32, i64, p, i32, p, i64, cint, f32, p, p, p, p, i64, p]
        L.moe_balance_loss_backward.argtypes = [p, cint, i64, i32, i64, p, i32, p, i64, cint, p, p, p, i64, p]
        L.moe_balance_workspace_bytes.restype = i64
        for name in ("moe_dispatch", "moe_balance_loss", "moe_balance_loss_backward"):
            getattr(L, name).restype = cint
        _lib = L
    return _lib


def _ids(ids: torch.Tensor, tokens=None):
    if ids.dtype != torch.int32 or ids.dim() != 2 or not ids.is_contiguous():
        raise Fp8qError("ids must be a contiguous int32 [tokens][topk] tensor")
    if tokens is not None and ids.shape[0] != tokens:
        raise Fp8qError("ids and logits disagree on the tokens (%d vs %d)" % (ids.shape[0], tokens))


def _workspace(workspace, nbytes: int, device, stream) -> torch.Tensor:
    if workspace is None:
        return _new(nbytes, torch.uint8, device, stream)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise Fp8qError("workspace must be a contiguous uint8 tensor")
    return workspace


def _array(t, shape, dtype, device, stream, name: str) -> torch.Tensor:
    """A contiguous output array: new when absent, checked otherwise."""
    if t is None:
        return _new(shape, dtype, device, stream)
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t
    _check_tensor(t, shape, (dtype,), name)
    if not t.is_contiguous():
        raise Fp8qError("%s must be contiguous" % name)
    return t


def _layout_args(experts: int, align: int, first: int) -> None:
    """The C call takes these as 32 bits, and ctypes would drop the others."""
    if not 1 <= experts <= MOE_MAX_EXPERTS:
        raise Fp8qError("experts must be 1..%d, got %d" % (MOE_MAX_EXPERTS, experts))
    if not 1 <= align <= 0x7FFFFFFF or not 0 <= first <= 0x7FFFFFFF - experts:
        raise Fp8qError("align = %d or first = %d is out of range" % (align, first))


def moe_dispatch(ids: torch.Tensor, experts: int, align: int = 128, first: int = 0,
                 group_offsets: torch.Tensor | None = None, group_rows: torch.Tensor | None = None,
                 dst_rows: torch.Tensor | None = None, stream=None, workspace: torch.Tensor | None = None):
    """The expert-sorted row layout of the routes ``ids`` (int32
    ``[tokens][topk]``, topk 1..8) to experts ``[first, first + experts)``;
    other ids (a dropped route, another rank's expert) are no route.

    Returns ``group_offsets[experts + 1]`` (segments of whole multiples of
    ``align`` rows), ``group_rows[experts]`` (the per-expert counts) and
    ``dst_rows[tokens][topk]`` (the row of each route, in token order inside
    its expert; -1 for none), all int32: the arguments of the scattering
    quantizers and the grouped GEMMs. A layout never takes more than ``tokens *
    topk + experts * (align - 1)`` rows.
    """
    dev = _on_gpu(ids, group_offsets, group_rows, dst_rows, workspace)
    _ids(ids)
    _layout_args(experts, align, first)
    tokens, topk = ids.shape
    group_offsets = _array(group_offsets, (experts + 1,), torch.int32, dev, stream, "group_offsets")
    group_rows = _array(group_rows, (experts,), torch.int32, dev, stream, "group_rows")
    dst_rows = _array(dst_rows, (tokens, topk), torch.int32, dev, stream, "dst_rows")
    workspace = _workspace(workspace, MOE_DISPATCH_WORKSPACE_BYTES, dev, stream)
    st = _call(_library().moe_dispatch, dev, stream, ids.data_ptr(), tokens, topk, first, experts, align,
               group_offsets.data_ptr(), group_rows.data_ptr(), dst_rows.data_ptr(), workspace.data_ptr(),
               workspace.numel())
    _check(st, "moe_dispatch")
    return group_offsets, group_rows, dst_rows


_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}
_LOGITS = {torch.bfloat16: LOGITS_BF16, torch.float32: LOGITS_F32}


def _balance_args(logits, ids, seq_offsets, score):
    """Checked leading arguments of the two balance entry points."""
    if logits.dtype not in _LOGITS:
        raise Fp8qError("logits must be bfloat16 or float32")
    if logits.dim() != 2 or (logits.numel() > 0 and (logits.stride(1) != 1 or logits.stride(0) < 0)):
        raise Fp8qError("logits must be [tokens][experts] with unit column stride")
    tokens, experts = logits.shape
    _ids(ids, tokens)
    if seq_offsets is not None and (seq_offsets.dtype != torch.int32 or seq_offsets.dim() != 1
                                    or seq_offsets.numel() < 2 or not seq_offsets.is_contiguous()):
        raise Fp8qError("seq_offsets must be a contiguous int32 tensor of S + 1 >= 2 entries")
    if score not in _SCORES:
        raise Fp8qError("score must be 'softmax' or 'sigmoid'")
    seqs = 1 if seq_offsets is None else seq_offsets.numel() - 1
    ld = experts if tokens <= 1 else logits.stride(0)
    return (logits.data_ptr(), _LOGITS[logits.dtype], tokens, experts, ld, ids.data_ptr(), ids.shape[1],
            _address(seq_offsets), seqs, _SCORES[score])


def moe_balance_loss(logits: torch.Tensor, ids: torch.Tensor, seq_offsets: torch.Tensor | None = None,
                     score: str = "softmax", alpha: float = 1.0, loss: torch.Tensor | None = None,
                     counts: torch.Tensor | None = None, coef: torch.Tensor | None = None, stream=None,
                     workspace: torch.Tensor | None = None):
    """Balance loss ``alpha * mean over sequences of sum_e f_e P_e`` of router
    ``logits`` (bf16 or fp32 ``[tokens][experts]``) and chosen experts ``ids``
    (int32 ``[tokens][topk]``, an id outside the experts is no route, a token
    without a route is not counted).

    ``f_e``: the expert's share of the routes times the number of experts;
    ``P_e``: the mean score of the counted tokens; ``score``: ``"softmax"`` or
    ``"sigmoid"`` (normalised over the experts). ``seq_offsets``: int32
    ``[S + 1]`` cuts the tokens into sequences, whose losses are averaged; None:
    one. Returns ``(loss[1], counts[S][experts], coef[S][experts])``; pass
    ``coef`` to :func:`moe_balance_loss_backward`. As everywhere in this package
    there is no autograd: the loss has no graph, also where ``logits`` requires a
    gradient, and adding it to a model's loss trains nothing by itself.
    """
    dev = _on_gpu(logits, ids, seq_offsets, loss, counts, coef, workspace)
    args = _balance_args(logits, ids, seq_offsets, score)
    tokens, experts, seqs = args[2], args[3], args[8]
    loss = _array(loss, (1,), torch.float32, dev, stream, "loss")
    counts = _array(counts, (seqs, experts), torch.int32, dev, stream, "counts")
    coef = _array(coef, (seqs, experts), torch.float32, dev, stream, "coef")
    lib = _library()
    workspace = _workspace(workspace, lib.moe_balance_workspace_bytes(tokens, experts, seqs), dev, stream)
    st = _call(lib.moe_balance_loss, dev, stream, *args, float(alpha), loss.data_ptr(), counts.data_ptr(),
               coef.data_ptr(), workspace.data_ptr(), workspace.numel())
    _check(st, "moe_balance_loss")
    return loss, counts, coef


def moe_balance_loss_backward(logits: torch.Tensor, ids: torch.Tensor, coef: torch.Tensor,
                              grad: torch.Tensor | None = None, seq_offsets: torch.Tensor | None = None,
                              score: str = "softmax", out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of :func:`moe_balance_loss` with respect to the logits, in the
    logits' dtype. ``coef`` is what the forward call returned; ``grad``: the
    loss's own gradient (one fp32 element; None: 1). ``out`` may be ``logits``.
    """
    dev = _on_gpu(logits, ids, coef, grad, seq_offsets, out)
    args = _balance_args(logits, ids, seq_offsets, score)
    tokens, experts, seqs = args[2], args[3], args[8]
    _array(coef, (seqs, experts), torch.float32, dev, stream, "coef")
    if grad is not None and (grad.dtype != torch.float32 or grad.numel() != 1):
        raise Fp8qError("grad must hold one float32 element")
    if out is None:
        out = _new((tokens, experts), logits.dtype, dev, stream)
    else:
        _check_tensor(out, (tokens, experts), (logits.dtype,), "out")
    st = _call(_library().moe_balance_loss_backward, dev, stream, *args, coef.data_ptr(), _address(grad),
               out.data_ptr(), experts if tokens <= 1 else out.stride(0))
    _check(st, "moe_balance_loss_backward")
    return out
