"""CPU checks of the MoE entry points: exported symbols, limits, status codes
of calls that the host refuses before any launch, the binding's own checks."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from fine_grained_fp8_quantize_amd import _moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ENUM = 0, 1, 2, 3, 4
A, B, C, D, W = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


def _lib():
    if not os.path.exists(fq.library_path()):
        from fine_grained_fp8_quantize_amd import build
        build.build(force=False)
    return _moe._library()


def test_header_is_exported_and_its_limits_are_the_bindings():
    text = open(os.path.join(ROOT, "include", "fp8q_moe.h")).read()
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", code, flags=re.M)
    assert sorted(names) == ["moe_balance_loss", "moe_balance_loss_backward", "moe_balance_workspace_bytes",
                             "moe_dispatch"]
    _lib()
    raw = ctypes.CDLL(fq.library_path())
    assert all(hasattr(raw, n) for n in names)
    limits = dict(re.findall(r"#define\s+FP8Q_(\w+)\s+(\d+)", code))
    for name in ("MOE_MAX_EXPERTS", "MOE_MAX_TOPK", "MOE_DISPATCH_WORKSPACE_BYTES", "SCORE_SOFTMAX", "SCORE_SIGMOID",
                 "LOGITS_BF16", "LOGITS_F32"):
        assert int(limits[name]) == getattr(_moe, name), name


def _d(ids=A, tokens=10, topk=2, first=0, experts=8, align=16, off=B, rows=C, dst=D, ws=W, n=262144):
    return _lib().moe_dispatch(ids, tokens, topk, first, experts, align, off, rows, dst, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), ERR_SHAPE), (dict(topk=0), ERR_SHAPE), (dict(topk=9), ERR_SHAPE), (dict(experts=0), ERR_SHAPE),
    (dict(experts=1025), ERR_SHAPE), (dict(align=0), ERR_SHAPE), (dict(first=-1), ERR_SHAPE),
    (dict(first=0x7FFFFFFF), ERR_SHAPE), (dict(tokens=1 << 30, topk=2), ERR_SHAPE), (dict(n=262143), ERR_SHAPE),
    (dict(align=1 << 30), ERR_SHAPE), (dict(ids=0), ERR_NULL), (dict(off=0), ERR_NULL), (dict(rows=0), ERR_NULL),
    (dict(dst=0), ERR_NULL), (dict(ws=0), ERR_NULL), (dict(ids=A + 2), ERR_ALIGN), (dict(ws=W + 1), ERR_ALIGN)])
def test_dispatch_refusals(kw, want):
    assert _d(**kw) == want


def _f(logits=A, dt=1, tokens=10, experts=8, ld=8, ids=B, topk=2, off=C, seqs=3, score=0, loss=D, counts=D, coef=D,
       ws=W, n=1 << 20):
    return _lib().moe_balance_loss(logits, dt, tokens, experts, ld, ids, topk, off, seqs, score, 1.0, loss, counts,
                                   coef, ws, n, None)


BOTH = [(dict(dt=2), ERR_ENUM), (dict(score=2), ERR_ENUM), (dict(tokens=-1), ERR_SHAPE), (dict(experts=0), ERR_SHAPE),
        (dict(experts=1025, ld=1025), ERR_SHAPE), (dict(topk=0), ERR_SHAPE), (dict(topk=9), ERR_SHAPE),
        (dict(seqs=0), ERR_SHAPE), (dict(seqs=32769), ERR_SHAPE), (dict(ld=7), ERR_SHAPE), (dict(off=0), ERR_NULL), (dict(logits=0), ERR_NULL),
        (dict(ids=0), ERR_NULL), (dict(coef=0), ERR_NULL), (dict(logits=A + 2), ERR_ALIGN), (dict(ids=B + 1), ERR_ALIGN),
        (dict(off=C + 2), ERR_ALIGN), (dict(logits=A + 1, dt=0), ERR_ALIGN)]


@pytest.mark.parametrize("kw,want", BOTH + [(dict(loss=0), ERR_NULL), (dict(counts=0), ERR_NULL), (dict(ws=0), ERR_NULL),
                                            (dict(n=100), ERR_SHAPE), (dict(loss=D + 2), ERR_ALIGN)])
def test_balance_refusals(kw, want):
    assert _f(**kw) == want


def _b(logits=A, dt=1, tokens=10, experts=8, ld=8, ids=B, topk=2, off=C, seqs=3, score=0, coef=D, grad=D, out=W, ld_d=8):
    return _lib().moe_balance_loss_backward(logits, dt, tokens, experts, ld, ids, topk, off, seqs, score, coef, grad,
                                            out, ld_d, None)


@pytest.mark.parametrize("kw,want", BOTH + [(dict(out=0), ERR_NULL), (dict(ld_d=7), ERR_SHAPE), (dict(tokens=0), OK),
                                            (dict(out=W + 2), ERR_ALIGN), (dict(grad=D + 1), ERR_ALIGN),
                                            (dict(out=A, ld_d=9), ERR_SHAPE)])
def test_balance_backward_refusals(kw, want):
    assert _b(**kw) == want


def test_workspace_bytes():
    f = _lib().moe_balance_workspace_bytes
    assert f(-1, 8, 1) == 0 and f(1, 0, 1) == 0 and f(1, 2000, 1) == 0 and f(1, 8, 0) == 0 and f(1, 8, 32769) == 0
    assert 0 < f(0, 8, 1) <= f(100, 8, 1) < f(100, 8, 50) < f(100, 64, 50)
    assert f(1 << 30, 256, 1) < 8 << 20      # long batches are cut into no more parts


def test_binding_checks():
    ids, x = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 8))
    for call in (lambda: fq.moe_dispatch(ids, 8), lambda: fq.moe_balance_loss(x, ids),
                 lambda: fq.moe_balance_loss_backward(x, ids, torch.zeros((1, 8)))):
        with pytest.raises(fq.Fp8qError, match="GPU"):
            call()
    for bad in (dict(logits=x.half()), dict(logits=x.t()), dict(logits=x[0]), dict(ids=ids.long()), dict(ids=ids[:3]),
                dict(ids=ids[:, :1]), dict(seq_offsets=torch.zeros(1, dtype=torch.int32)), dict(score="max"),
                dict(seq_offsets=torch.zeros(3))):
        kw = {"logits": x, "ids": ids, "seq_offsets": None, "score": "softmax", **bad}
        with pytest.raises(fq.Fp8qError):
            _moe._balance_args(**kw)
