"""MoE routing operators (``include/fp8q_moe.h``): the binding of the
``moe_*`` entry points. Imported by the package; see its docstring."""
from __future__ import annotations

import ctypes

import torch

from . import Fp8qError, _check, _check_tensor, _empty, _load, _need_gpu, _ptr, _stream
from ._mx4 import _same_device

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
        return _empty((nbytes,), torch.uint8, device, stream)
    _need_gpu(workspace)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise Fp8qError("workspace must be a contiguous uint8 tensor")
    return workspace


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
    _need_gpu(ids, group_offsets, group_rows, dst_rows)
    _same_device(ids, group_offsets, group_rows, dst_rows, workspace)
    _ids(ids)
    tokens, topk = ids.shape
    dev = ids.device
    if group_offsets is None:
        group_offsets = _empty((experts + 1,), torch.int32, dev, stream)
    if group_rows is None:
        group_rows = _empty((experts,), torch.int32, dev, stream)
    if dst_rows is None:
        dst_rows = _empty((tokens, topk), torch.int32, dev, stream)
    _check_tensor(group_offsets, (experts + 1,), (torch.int32,), "group_offsets")
    _check_tensor(group_rows, (experts,), (torch.int32,), "group_rows")
    _check_tensor(dst_rows, (tokens, topk), (torch.int32,), "dst_rows")
    if not dst_rows.is_contiguous():
        raise Fp8qError("dst_rows must be contiguous [tokens][topk]")
    workspace = _workspace(workspace, MOE_DISPATCH_WORKSPACE_BYTES, dev, stream)
    st = _library().moe_dispatch(_ptr(ids), tokens, topk, first, experts, align, _ptr(group_offsets),
                                 _ptr(group_rows), _ptr(dst_rows), _ptr(workspace), workspace.numel(),
                                 _stream(stream))
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
    return (_ptr(logits), _LOGITS[logits.dtype], tokens, experts, ld, _ptr(ids), ids.shape[1], _ptr(seq_offsets),
            seqs, _SCORES[score])


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
    ``coef`` to :func:`moe_balance_loss_backward`.
    """
    _need_gpu(logits, ids, seq_offsets, loss, counts, coef)
    _same_device(logits, ids, seq_offsets, loss, counts, coef, workspace)
    args = _balance_args(logits, ids, seq_offsets, score)
    tokens, experts, seqs = args[2], args[3], args[8]
    dev = logits.device
    if loss is None:
        loss = _empty((1,), torch.float32, dev, stream)
    if counts is None:
        counts = _empty((seqs, experts), torch.int32, dev, stream)
    if coef is None:
        coef = _empty((seqs, experts), torch.float32, dev, stream)
    _check_tensor(loss, (1,), (torch.float32,), "loss")
    for t, dt, name in ((counts, torch.int32, "counts"), (coef, torch.float32, "coef")):
        _check_tensor(t, (seqs, experts), (dt,), name)
        if not t.is_contiguous():
            raise Fp8qError("%s must be contiguous" % name)
    lib = _library()
    workspace = _workspace(workspace, lib.moe_balance_workspace_bytes(tokens, experts, seqs), dev, stream)
    st = lib.moe_balance_loss(*args, float(alpha), _ptr(loss), _ptr(counts), _ptr(coef), _ptr(workspace),
                              workspace.numel(), _stream(stream))
    _check(st, "moe_balance_loss")
    return loss, counts, coef


def moe_balance_loss_backward(logits: torch.Tensor, ids: torch.Tensor, coef: torch.Tensor,
                              grad: torch.Tensor | None = None, seq_offsets: torch.Tensor | None = None,
                              score: str = "softmax", out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of :func:`moe_balance_loss` with respect to the logits, in the
    logits' dtype. ``coef`` is what the forward call returned; ``grad``: the
    loss's own gradient (one fp32 element; None: 1). ``out`` may be ``logits``.
    """
    _need_gpu(logits, ids, coef, grad, seq_offsets, out)
    _same_device(logits, ids, coef, grad, seq_offsets, out)
    args = _balance_args(logits, ids, seq_offsets, score)
    tokens, experts, seqs = args[2], args[3], args[8]
    _check_tensor(coef, (seqs, experts), (torch.float32,), "coef")
    if not coef.is_contiguous():
        raise Fp8qError("coef must be contiguous")
    if grad is not None and (grad.dtype != torch.float32 or grad.numel() != 1):
        raise Fp8qError("grad must hold one float32 element")
    if out is None:
        out = _empty((tokens, experts), logits.dtype, logits.device, stream)
    _check_tensor(out, (tokens, experts), (logits.dtype,), "out")
    st = _library().moe_balance_loss_backward(*args, _ptr(coef), _ptr(grad), _ptr(out),
                                              experts if tokens <= 1 else out.stride(0), _stream(stream))
    _check(st, "moe_balance_loss_backward")
    return out
