"""CPU checks of the FP4 entry points: exported symbols, status codes of calls
that the host refuses before any launch, and the binding's own checks."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from fine_grained_fp8_quantize_amd import _mx4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ENUM = 0, 1, 2, 3, 4
# well-aligned made-up addresses: validation reads no memory
X, Q, S, Y, D = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


def _lib():
    if not os.path.exists(fq.library_path()):
        from fine_grained_fp8_quantize_amd import build
        build.build(force=False)
    return _mx4._library()


def test_header_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8q_mx4.h")).read(), flags=re.S)
    names = re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M)
    assert len(names) == 5
    _lib()
    raw = ctypes.CDLL(fq.library_path())
    for name in names:
        assert hasattr(raw, name) and callable(getattr(fq, name)) and name in fq.__all__, name


def _q(groups=2, x=X, rows=40, cols=600, ld_x=600, sx=24000, tiling=0, q=Q, ld_q=3, sq=15360, s=S, ld_s=3, ss=384):
    return _lib().fp4_quantize_mx(groups, x, rows, cols, ld_x, sx, tiling, q, ld_q, sq, s, ld_s, ss, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tiling=2), ERR_ENUM), (dict(tiling=-1), ERR_ENUM), (dict(groups=-1), ERR_SHAPE), (dict(rows=-1), ERR_SHAPE),
    (dict(cols=-1), ERR_SHAPE), (dict(cols=1 << 41), ERR_SHAPE), (dict(groups=0), OK), (dict(rows=0), OK),
    (dict(cols=0), OK), (dict(x=0), ERR_NULL), (dict(q=0), ERR_NULL), (dict(s=0), ERR_NULL),
    (dict(ld_x=599), ERR_SHAPE), (dict(ld_q=2), ERR_SHAPE), (dict(ld_s=2), ERR_SHAPE), (dict(sx=-1), ERR_SHAPE),
    (dict(sq=15344), ERR_SHAPE), (dict(ss=383), ERR_SHAPE), (dict(sq=15368), ERR_ALIGN), (dict(q=Q + 8), ERR_ALIGN),
    (dict(s=S + 2), ERR_ALIGN), (dict(x=X + 1), ERR_ALIGN), (dict(ld_q=1 << 41), ERR_SHAPE),
    (dict(sx=1 << 62), ERR_SHAPE), (dict(ld_x=1 << 60), ERR_SHAPE),
    # transposed: 38 row tiles
    (dict(tiling=1), ERR_SHAPE)])
def test_quantize_refusals(kw, want):
    assert _q(**kw) == want


def _sc(x=X, tokens=5, cols=200, ld_x=200, topk=2, dst=D, m=64, q=Q, ld_q=4, s=S, ld_s=4):
    return _lib().fp4_quantize_mx_scatter(x, tokens, cols, ld_x, topk, dst, m, q, ld_q, s, ld_s, None)


@pytest.mark.parametrize("kw,want", [
    (dict(topk=0), ERR_SHAPE), (dict(topk=9), ERR_SHAPE), (dict(tokens=-1), ERR_SHAPE), (dict(m=-1), ERR_SHAPE),
    (dict(tokens=0), OK), (dict(cols=0), OK), (dict(m=0), OK), (dict(x=0), ERR_NULL), (dict(dst=0), ERR_NULL),
    (dict(q=0), ERR_NULL), (dict(ld_x=199), ERR_SHAPE), (dict(ld_q=3), ERR_SHAPE), (dict(ld_s=3), ERR_SHAPE),
    (dict(dst=D + 2), ERR_ALIGN), (dict(q=Q + 4), ERR_ALIGN)])
def test_scatter_refusals(kw, want):
    assert _sc(**kw) == want


def _dq(q=Q, ld_q=3, s=S, ld_s=3, rows=40, cols=600, y=Y, ld_y=600, dt=0):
    return _lib().fp4_dequantize_mx(q, ld_q, s, ld_s, rows, cols, y, ld_y, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), ERR_ENUM), (dict(rows=-1), ERR_SHAPE), (dict(rows=0), OK), (dict(cols=0), OK), (dict(q=0), ERR_NULL),
    (dict(s=0), ERR_NULL), (dict(y=0), ERR_NULL), (dict(ld_y=599), ERR_SHAPE), (dict(ld_q=2), ERR_SHAPE),
    (dict(y=Y + 1), ERR_ALIGN), (dict(y=Y + 2, dt=1), ERR_ALIGN), (dict(q=Q + 4), ERR_ALIGN)])
def test_dequantize_refusals(kw, want):
    assert _dq(**kw) == want


def _g(m=40, n=50, k=600, a=X, ld_a=3, sa=S, ld_as=3, b=Q, ld_b=4, sb=S, ld_bs=4, c=Y, ldc=50, dt=0):
    return _lib().fp4_gemm_mx(m, n, k, a, ld_a, sa, ld_as, b, ld_b, sb, ld_bs, c, ldc, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=3), ERR_ENUM), (dict(m=-1), ERR_SHAPE), (dict(n=-1), ERR_SHAPE), (dict(k=-1), ERR_SHAPE),
    (dict(m=0), OK), (dict(n=0), OK), (dict(a=0), ERR_NULL), (dict(sa=0), ERR_NULL), (dict(b=0), ERR_NULL),
    (dict(sb=0), ERR_NULL), (dict(c=0), ERR_NULL), (dict(c=0, k=0), ERR_NULL), (dict(ld_a=2), ERR_SHAPE),
    (dict(ld_as=2), ERR_SHAPE), (dict(ld_b=3), ERR_SHAPE), (dict(ld_bs=3), ERR_SHAPE), (dict(ldc=49), ERR_SHAPE),
    (dict(a=X + 8), ERR_ALIGN), (dict(b=Q + 8), ERR_ALIGN), (dict(sa=S + 1), ERR_ALIGN), (dict(c=Y + 1), ERR_ALIGN),
    (dict(c=Y + 2, dt=1), ERR_ALIGN), (dict(m=1 << 39, ld_a=1 << 39, ld_as=1 << 39, n=1 << 39), ERR_SHAPE)])
def test_gemm_refusals(kw, want):
    assert _g(**kw) == want


def _gg(groups=3, off=D, rows=D, m=64, n=50, k=600, a=X, ld_a=4, sa=S, ld_as=4, b=Q, ld_b=4, stb=20480, sb=S, ld_bs=4,
        sts=512, c=Y, ldc=50, dt=0):
    return _lib().fp4_grouped_gemm_mx(groups, off, rows, m, n, k, a, ld_a, sa, ld_as, b, ld_b, stb, sb, ld_bs, sts, c,
                                      ldc, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=9), ERR_ENUM), (dict(groups=-1), ERR_SHAPE), (dict(groups=0), OK), (dict(m=0), OK), (dict(n=0), OK),
    (dict(off=0), ERR_NULL), (dict(a=0), ERR_NULL), (dict(c=0), ERR_NULL), (dict(m=72, ld_a=5, ld_as=5), ERR_SHAPE),
    (dict(stb=-16), ERR_SHAPE), (dict(sts=-1), ERR_SHAPE), (dict(ldc=49), ERR_SHAPE), (dict(stb=20488), ERR_ALIGN),
    (dict(off=D + 2), ERR_ALIGN), (dict(rows=D + 1), ERR_ALIGN), (dict(m=1 << 31, ld_a=1 << 27, ld_as=1 << 27), ERR_SHAPE)])
def test_grouped_refusals(kw, want):
    assert _gg(**kw) == want


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((16, 128), dtype=torch.bfloat16)
    q, s = torch.zeros((1, 1, 1024), dtype=torch.uint8), torch.zeros((1, 1, 64), dtype=torch.int32)
    for call in (lambda: fq.fp4_quantize_mx(x), lambda: fq.fp4_dequantize_mx(q, s, 16, 128),
                 lambda: fq.fp4_gemm_mx(q, s, q, s),
                 lambda: fq.fp4_quantize_mx_scatter(x, torch.zeros((16, 1), dtype=torch.int32), 16),
                 lambda: fq.fp4_grouped_gemm_mx(torch.zeros(2, dtype=torch.int32), None, q, s, q[None], s[None])):
        with pytest.raises(fq.Fp8qError, match="GPU"):
            call()


def test_binding_checks_a_matrix_of_tiles():
    q, s = torch.zeros((5, 3, 1024), dtype=torch.uint8), torch.zeros((2, 3, 64), dtype=torch.int32)
    assert _mx4._matrix(q, s, "q") == (5, 3, 3, 3)
    assert _mx4._matrix(q[:, 1:2], s[:, 1:2], "q") == (5, 1, 3, 3)        # a range of row tiles
    assert _mx4._matrix(torch.stack((q, q)), torch.stack((s, s)), "q", 1) == (5, 3, 3, 3)
    for bad_q, bad_s in ((q.to(torch.int8), s), (q, s[:1]), (q[..., :512], s), (q[:, :2], s), (q, s.float()),
                         (q.transpose(1, 2).contiguous().transpose(1, 2), s), (q[0], s)):
        with pytest.raises(fq.Fp8qError):
            _mx4._matrix(bad_q, bad_s, "q")


def test_row_counts_fit_the_tiles():
    assert _mx4._rows_of(None, 3, "m") == 48
    assert _mx4._rows_of(33, 3, "m") == 33
    for rows in (32, 49, 0):
        with pytest.raises(fq.Fp8qError):
            _mx4._rows_of(rows, 3, "m")
