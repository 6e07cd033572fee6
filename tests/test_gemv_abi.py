"""CPU checks of the weight-only FP4 entry points: exported symbols, status
codes of calls that the host refuses before any launch."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

import fine_grained_fp8_quantize_amd as fq
from fine_grained_fp8_quantize_amd import _gemv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ENUM = 0, 1, 2, 3, 4
X, W, S, Y, I = (0x10000 * i for i in range(1, 6))


def _lib():
    if not os.path.exists(fq.library_path()):
        from fine_grained_fp8_quantize_amd import build
        build.build(force=False)
    return _gemv._library()


def test_header_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "fp8q_gemv.h")).read()
    names = re.findall(r"^\s*int\s+(\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S), flags=re.M)
    assert names == ["fp4_gemv_mx", "fp4_gated_gemv_mx"]
    _lib()
    raw = ctypes.CDLL(fq.library_path())
    for name in names:
        assert hasattr(raw, name) and callable(getattr(fq, name)) and name in fq.__all__, name


def _v(tokens=5, topk=1, ids=0, first=0, experts=1, n=40, k=600, x=X, ld_x=600, ld_xj=0, w=W, ld_w=3, sw=15360, s=S, ld_s=3,
       ss=384, y=Y, ld_y=40, dt=0):
    return _lib().fp4_gemv_mx(tokens, topk, ids, first, experts, n, k, x, ld_x, ld_xj, w, ld_w, sw, s, ld_s, ss, y, ld_y, dt,
                              None)


R = dict(ids=I, topk=3, experts=4)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), ERR_ENUM), (dict(dt=-1), ERR_ENUM), (dict(tokens=-1), ERR_SHAPE), (dict(topk=-1), ERR_SHAPE),
    (dict(n=-1), ERR_SHAPE), (dict(k=-1), ERR_SHAPE), (dict(tokens=0), OK), (dict(n=0), OK), (dict(topk=0), OK),
    (dict(x=0), ERR_NULL), (dict(w=0), ERR_NULL), (dict(s=0), ERR_NULL), (dict(y=0), ERR_NULL), (dict(ld_w=2), ERR_SHAPE),
    (dict(ld_s=2), ERR_SHAPE), (dict(ld_y=39), ERR_SHAPE), (dict(ld_x=-1), ERR_SHAPE), (dict(ld_xj=-8), ERR_SHAPE),
    (dict(sw=-16), ERR_SHAPE), (dict(ss=-1), ERR_SHAPE), (dict(sw=24), ERR_ALIGN), (dict(w=W + 8), ERR_ALIGN),
    (dict(s=S + 2), ERR_ALIGN), (dict(x=X + 1), ERR_ALIGN), (dict(y=Y + 1), ERR_ALIGN), (dict(y=Y + 2, dt=1), ERR_ALIGN),
    (dict(topk=2), ERR_SHAPE), (dict(experts=2), ERR_SHAPE), (dict(tokens=64 * 65535 + 1), ERR_SHAPE),
    (dict(n=1 << 31, ld_y=1 << 31), ERR_SHAPE), (dict(k=1 << 38), ERR_SHAPE), (dict(ld_y=1 << 61), ERR_SHAPE),
    (dict(ld_x=1 << 61), ERR_SHAPE), (dict(ld_w=1 << 41), ERR_SHAPE), (dict(R, ids=I + 2), ERR_ALIGN),
    (dict(R, topk=33), ERR_SHAPE), (dict(R, tokens=2000), ERR_SHAPE), (dict(R, experts=-1), ERR_SHAPE), (dict(R, experts=0, y=0), ERR_NULL),
    (dict(R, experts=1025), ERR_SHAPE), (dict(R, first=-1), ERR_SHAPE), (dict(R, first=0x7FFFFFFE), ERR_SHAPE),
    (dict(R, tokens=0), OK), (dict(R, sw=1 << 60), ERR_SHAPE)])
def test_refusals(kw, want):
    assert _v(**kw) == want


def _g(act=0, su=7680, sus=192, dt=0, n=40, w=W):
    return _lib().fp4_gated_gemv_mx(5, 1, 0, 0, 1, n, 600, X, 600, 0, w, 3, su, 0, S, 3, sus, 0, act, Y, 40, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(act=2), ERR_ENUM), (dict(act=-1), ERR_ENUM), (dict(dt=5), ERR_ENUM), (dict(su=-16), ERR_SHAPE),
    (dict(sus=-1), ERR_SHAPE), (dict(su=8), ERR_ALIGN), (dict(su=1 << 61), ERR_SHAPE), (dict(n=41), ERR_SHAPE),
    (dict(w=0), ERR_NULL)])
def test_gated_refusals(kw, want):
    assert _g(**kw) == want
