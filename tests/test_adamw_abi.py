"""CPU checks of the optimizer's entry point: the exported symbol, the status
codes of calls that the host refuses before any launch, and the CPU model
against the formula."""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest

import fine_grained_fp8_quantize_amd as fq
from fine_grained_fp8_quantize_amd import _adamw
from oracle import adamw as model

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ENUM = 0, 1, 2, 3, 4


def _lib():
    if not os.path.exists(fq.library_path()):
        from fine_grained_fp8_quantize_amd import build
        build.build(force=False)
    return _adamw._library()


def test_header_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "fp8q_adamw.h")).read(), flags=re.S)
    assert re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M) == ["adamw_step"]
    _lib()
    assert hasattr(ctypes.CDLL(fq.library_path()), "adamw_step")
    for name in ("adamw_plan", "adamw_step"):
        assert callable(getattr(fq, name)) and name in fq.__all__
    fields = re.findall(r"(\w+);", text[text.index("typedef struct"):text.index("} fp8q_adamw_tensor")])
    assert fields == [f for f, _ in _adamw._Tensor._fields_]


def _step(count=1, tensors=None, pd=1, gd=0, bits=32, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=1, lr_dev=0,
          step_dev=0, scale=0, null=False,
          no_grads=False, **entry):
    """A call whose one tensor is empty, unless `entry` gives it elements: nothing is ever launched."""
    e = (_adamw._Tensor * 1)()
    grad = entry.pop("grad", 0x2000)
    fields = dict(param=0x1000, exp_avg=0x3000, exp_avg_sq=0x4000, copy=0x5000, numel=0)
    if bits == 8:
        fields.update(exp_avg_scale=0x6000, exp_avg_sq_scale=0x7000)
    for k, v in {**fields, **entry}.items():
        setattr(e[0], k, v)
    g = (ctypes.c_void_p * 1)(grad)
    return _lib().adamw_step(count, None if null else e, None if no_grads else g, pd, gd, bits, lr, b1, b2, eps, wd, step, lr_dev, step_dev, scale, 0,
                             None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(count=0, null=True), OK), (dict(numel=5, grad=0), OK), (dict(null=True), ERR_NULL),
    (dict(no_grads=True), ERR_NULL),
    (dict(pd=2), ERR_ENUM), (dict(gd=-1), ERR_ENUM), (dict(bits=16), ERR_ENUM), (dict(count=-1), ERR_SHAPE),
    (dict(step=0), ERR_SHAPE), (dict(step=0, step_dev=0x100), OK), (dict(step_dev=0x104), ERR_ALIGN),
    (dict(lr_dev=0x102), ERR_ALIGN), (dict(scale=0x101), ERR_ALIGN), (dict(b1=1.0), ERR_SHAPE),
    (dict(b1=-0.1), ERR_SHAPE), (dict(b2=1.5), ERR_SHAPE), (dict(b2=NAN), ERR_SHAPE), (dict(eps=-1.0), ERR_SHAPE),
    (dict(eps=INF), ERR_SHAPE), (dict(lr=NAN), ERR_SHAPE), (dict(wd=INF), ERR_SHAPE), (dict(numel=-1), ERR_SHAPE),
    (dict(numel=1 << 41), ERR_SHAPE), (dict(numel=5, param=0), ERR_NULL), (dict(numel=5, exp_avg=0), ERR_NULL),
    (dict(numel=5, exp_avg_sq=0), ERR_NULL), (dict(numel=5, bits=8, exp_avg_scale=0), ERR_NULL),
    (dict(numel=5, bits=8, exp_avg_sq_scale=0), ERR_NULL), (dict(numel=5, exp_avg_scale=0x6000), ERR_NULL),
    (dict(numel=5, pd=0), ERR_ENUM), (dict(numel=5, param=0x1002), ERR_ALIGN), (dict(numel=5, grad=0x2001), ERR_ALIGN),
    (dict(numel=5, gd=1, grad=0x2002), ERR_ALIGN), (dict(numel=5, exp_avg=0x3002), ERR_ALIGN),
    (dict(numel=5, bits=8, exp_avg_sq_scale=0x7002), ERR_ALIGN), (dict(numel=5, copy=0x5001), ERR_ALIGN)])
def test_refusals(kw, want):
    assert _step(**kw) == want


def test_the_model_follows_the_formula():
    """Every rounding is 2^-24: m at most 4 on either of its terms, the parameter 3 on itself and the update and
    15 on the update (its own 11 and m's 4)."""
    rng = np.random.default_rng(0)
    p, g, m = (rng.standard_normal(4000).astype(np.float32) * s for s in (0.02, 1e-3, 1e-3))
    v = (rng.standard_normal(4000).astype(np.float32) * np.float32(1e-3)) ** 2
    p, g, m = (x.astype(np.float32) for x in (p, g, m))
    h = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=7)
    a, b = model.step32(p, g, m, v, **h), model.step64(p, g, m, v, **h)
    u, terms = 2.0 ** -24, 0.9 * np.abs(m.astype(np.float64)) + 0.1 * np.abs(g.astype(np.float64))
    assert np.all(np.abs(a[1] - b[1]) <= 4.01 * u * terms) and np.all(np.abs(a[3] - b[2]) <= 6.01 * u * b[2])
    size = terms * h["lr"] / (1 - 0.9 ** 7) / (np.sqrt(b[2] / (1 - 0.95 ** 7)) + 1e-8)
    assert np.all(np.abs(a[0] - b[0]) <= u * (3.01 * (np.abs(p) + size) + 15.02 * size))


def test_the_models_codes():
    """Every code is a fixed point; between two codes, 16 random bits of zero give the lower one, all ones the upper
    one except within 2^-16 of the lower."""
    codes = np.arange(127, dtype=np.uint8)
    values = model.decode_e4m3(codes)
    for bits in (0, 1, 0xFFFF):
        assert np.array_equal(model.stochastic_e4m3(values, np.full(127, bits)), codes)
    mid = ((values[1:].astype(np.float64) + values[:-1]) / 2).astype(np.float32)
    assert np.array_equal(model.stochastic_e4m3(mid, np.full(126, 0x7FFF)), codes[:-1])
    assert np.array_equal(model.stochastic_e4m3(mid, np.full(126, 0x8000)), codes[1:])
    assert model.stochastic_e4m3(np.array([500.0]), np.array([0xFFFF]))[0] == 126
    bits = model.random_bits(1 << 20, 3, 5, 7).astype(np.int64)
    for half in (bits & 0xFFFF, bits >> 16):  # 16 buckets, 6 standard deviations of a binomial count
        n = np.bincount(half >> 12, minlength=16)
        assert np.all(np.abs(n - (1 << 16)) <= 6 * np.sqrt((1 << 20) / 16 * 15 / 16))
