"""CPU checks of the gated feed-forward entry points: exported symbols, status
codes of calls that the host refuses before any launch, the launch rules, and
the oracle's slopes against differences."""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest

import fine_grained_fp8_quantize_amd as fq
from fine_grained_fp8_quantize_amd import _gated
from oracle import gated as model

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ENUM = 0, 1, 2, 3, 4
A, AS, B, BS, C, CS, G, W, D = (0x10000 * i for i in range(1, 10))


def _lib():
    if not os.path.exists(fq.library_path()):
        from fine_grained_fp8_quantize_amd import build
        build.build(force=False)
    return _gated._library()


def test_header_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "fp8q_gated.h")).read()
    names = re.findall(r"^\s*int(?:64_t)?\s+(\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S), flags=re.M)
    assert len(names) == 5
    _lib()
    raw = ctypes.CDLL(fq.library_path())
    for name in names:
        assert hasattr(raw, name), name
        if not name.endswith("_bytes"):
            assert callable(getattr(fq, name)) and name in fq.__all__, name
    codes = dict(re.findall(r"#define\s+FP8Q_(\w+)\s+(\d+)", text))
    assert {k: int(v) for k, v in codes.items()} == {"ACT_SILU": _gated.ACT_SILU, "ACT_GELU": _gated.ACT_GELU,
                                                     "OUT_E4M3": _gated.OUT_E4M3}


def _g(m=40, n=256, k=512, a=A, lda=512, a_s=AS, ld_as=40, b=B, ldb=512, sb=131072, b_s=BS, ld_bs=4, sbs=8, act=0, out=C,
       ldo=256, dt=0, os_=0, ld_os=0, gu=0, ldg=0, ws=0, wsb=0):
    return _lib().fp8_gated_gemm(m, n, k, a, lda, a_s, ld_as, b, ldb, sb, b_s, ld_bs, sbs, act, out, ldo, dt, os_, ld_os,
                                 gu, ldg, ws, wsb, None)


E4 = dict(dt=2, os_=CS, ld_os=40)
GEMM = [
    (dict(act=2), ERR_ENUM), (dict(dt=3), ERR_ENUM), (dict(m=-1), ERR_SHAPE), (dict(n=-1), ERR_SHAPE),
    (dict(k=-128), ERR_SHAPE), (dict(m=0), OK), (dict(n=0), OK), (dict(a=0), ERR_NULL), (dict(a_s=0), ERR_NULL),
    (dict(b=0), ERR_NULL), (dict(b_s=0), ERR_NULL), (dict(out=0), ERR_NULL), (dict(k=500), ERR_SHAPE),
    (dict(lda=500), ERR_SHAPE), (dict(ldb=496), ERR_SHAPE), (dict(ld_as=39), ERR_SHAPE), (dict(ld_bs=3), ERR_SHAPE),
    (dict(sb=-16), ERR_SHAPE), (dict(sbs=-1), ERR_SHAPE), (dict(sbs=1 << 29), ERR_SHAPE), (dict(sb=8), ERR_ALIGN),
    (dict(lda=1 << 23), ERR_SHAPE), (dict(ldb=1 << 23), ERR_SHAPE), (dict(lda=520), ERR_ALIGN),
    (dict(a=A + 8), ERR_ALIGN), (dict(b=B + 4), ERR_ALIGN), (dict(a_s=AS + 2), ERR_ALIGN), (dict(b_s=BS + 1), ERR_ALIGN),
    (dict(out=C + 1), ERR_ALIGN), (dict(out=C + 2, dt=1), ERR_ALIGN), (dict(ldo=255), ERR_SHAPE), (dict(ws=W + 8, wsb=64), ERR_ALIGN),
    (dict(wsb=-1), ERR_SHAPE), (dict(gu=G, ldg=511), ERR_SHAPE), (dict(gu=G + 1, ldg=512), ERR_ALIGN),
    (dict(E4, out=C + 8), ERR_ALIGN), (dict(dt=2), ERR_NULL), (dict(E4, ld_os=39), ERR_SHAPE),
    (dict(E4, n=200), ERR_SHAPE), (dict(E4, ldo=264), ERR_ALIGN), (dict(E4, os_=CS + 2), ERR_ALIGN),
    (dict(m=1 << 39, n=1 << 39, ldo=1 << 39), ERR_SHAPE), (dict(m=1 << 41), ERR_SHAPE), (dict(ldo=1 << 60), ERR_SHAPE),
    (dict(m=1 << 36, ld_as=1 << 36), ERR_SHAPE),
    (dict(m=1, n=1 << 31, ldo=1 << 31, sbs=1 << 26, sb=1 << 41), ERR_SHAPE)]


@pytest.mark.parametrize("kw,want", GEMM)
def test_gemm_refusals(kw, want):
    assert _g(**kw) == want


def _gg(groups=3, off=D, rows=D + 64, m=384, n=256, k=512, a=A, lda=512, a_s=AS, ld_as=384, b=B, ldb=512, sb=131072,
        se=262144, b_s=BS, ld_bs=4, sbs=8, ses=16, act=0, out=C, ldo=256, dt=0, os_=0, ld_os=0, gu=0, ldg=0, ws=0, wsb=0):
    return _lib().fp8_grouped_gated_gemm(groups, off, rows, m, n, k, a, lda, a_s, ld_as, b, ldb, sb, se, b_s, ld_bs, sbs,
                                         ses, act, out, ldo, dt, os_, ld_os, gu, ldg, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(groups=0), OK), (dict(m=0), OK), (dict(n=0), OK), (dict(groups=-1), ERR_SHAPE), (dict(off=0), ERR_NULL),
    (dict(m=300), ERR_SHAPE), (dict(n=200, dt=2, os_=CS, ld_os=384), ERR_SHAPE), (dict(se=-16), ERR_SHAPE), (dict(ses=-1), ERR_SHAPE),
    (dict(se=24), ERR_ALIGN), (dict(off=D + 2), ERR_ALIGN), (dict(rows=D + 1), ERR_ALIGN), (dict(act=-1), ERR_ENUM),
    (dict(dt=9), ERR_ENUM), (dict(a=0), ERR_NULL), (dict(dt=2), ERR_NULL), (dict(ldo=248), ERR_SHAPE),
    (dict(m=1 << 31, ld_as=1 << 26), ERR_SHAPE), (dict(ws=W + 8, wsb=64), ERR_ALIGN), (dict(wsb=-1), ERR_SHAPE)])
def test_grouped_refusals(kw, want):
    assert _gg(**kw) == want


def _bw(m=256, n=128, dh=A, ld_dh=128, gu=B, ldg=256, act=0, dt=2, out=C, ldo=256, os_=CS, ld_os=256, t=G, ld_t=256,
        ts=W, ld_ts=256):
    return _lib().fp8_gated_backward(m, n, dh, ld_dh, gu, ldg, act, dt, out, ldo, os_, ld_os, t, ld_t, ts, ld_ts, None)


BF = dict(dt=0, os_=0, t=0, ts=0)


@pytest.mark.parametrize("kw,want", [
    (dict(act=2), ERR_ENUM), (dict(dt=1), ERR_ENUM), (dict(m=-1), ERR_SHAPE), (dict(m=0), OK), (dict(n=0), OK),
    (dict(dh=0), ERR_NULL), (dict(gu=0), ERR_NULL), (dict(out=0), ERR_NULL), (dict(os_=0), ERR_NULL),
    (dict(ts=0), ERR_NULL), (dict(ld_dh=120), ERR_SHAPE), (dict(ldg=248), ERR_SHAPE), (dict(ldo=240), ERR_SHAPE),
    (dict(ld_os=255), ERR_SHAPE), (dict(ld_t=240), ERR_SHAPE), (dict(ld_ts=255), ERR_SHAPE), (dict(n=100), ERR_SHAPE),
    (dict(m=200), ERR_SHAPE), (dict(dh=A + 2), ERR_ALIGN), (dict(gu=B + 8), ERR_ALIGN), (dict(out=C + 4), ERR_ALIGN),
    (dict(t=G + 8), ERR_ALIGN), (dict(ld_dh=132), ERR_ALIGN), (dict(ldg=260), ERR_ALIGN), (dict(ldo=264), ERR_ALIGN),
    (dict(ld_t=264), ERR_ALIGN), (dict(os_=CS + 1), ERR_ALIGN), (dict(ts=W + 2), ERR_ALIGN), (dict(BF, t=G), ERR_ENUM),
    (dict(BF, os_=CS), ERR_ENUM), (dict(BF, dh=A + 1), ERR_ALIGN), (dict(BF, m=1 << 39, n=1 << 20, ld_dh=1 << 20, ldg=1 << 21,
                                                                        ldo=1 << 21), ERR_SHAPE),
    (dict(BF, m=1 << 33, n=8), ERR_SHAPE)])
def test_backward_refusals(kw, want):
    assert _bw(**kw) == want


def test_workspace():
    L = _lib()
    assert L.fp8_gated_workspace_bytes(5, 256, 512) == 5 * 256 * 4
    assert L.fp8_gated_workspace_bytes(4096, 2048, 7168) == 0
    assert L.fp8_gated_workspace_bytes(-1, 256, 512) == 0
    assert L.fp8_grouped_gated_workspace_bytes(512, 256) == 512 * 256 * 4
    assert L.fp8_grouped_gated_workspace_bytes(8192, 2048) == 0
    assert L.fp8_grouped_gated_workspace_bytes(512, -1) == 0


def test_slopes_against_differences():
    g = np.linspace(-8, 8, 4001)
    for act in ("silu", "gelu"):
        d = (model.act(act, g + 1e-5) - model.act(act, g - 1e-5)) / 2e-5
        assert np.max(np.abs(d - model.slope(act, g))) < 1e-9


def test_the_oracles_codes():
    codes = np.arange(127, dtype=np.uint8)
    from oracle.adamw import decode_e4m3
    v = decode_e4m3(codes)
    assert np.array_equal(model.encode_e4m3(v), codes) and np.array_equal(model.encode_e4m3(-v), codes | 128)
    mid = (v[1:].astype(np.float64) + v[:-1]) / 2  # ties go to the even code
    assert np.array_equal(model.encode_e4m3(mid.astype(np.float32)), (codes[:-1] + 1) & 0xFE)
