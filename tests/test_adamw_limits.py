"""Limits of an optimizer step, which the host looks at before the first launch:
a tensor that no launch holds must not leave the tensors before it stepped."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

import fine_grained_fp8_quantize_amd as fq
from fine_grained_fp8_quantize_amd import _adamw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_SHAPE = 0, 2
MOST = (1 << 34) - 1024


def _step(sizes, grads, bits=32, eps=1e-8):
    """Tensors with a gradient are empty or too large: nothing is ever launched."""
    if not os.path.exists(fq.library_path()):
        from fine_grained_fp8_quantize_amd import build
        build.build(force=False)
    entries = (_adamw._Tensor * len(sizes))()
    for e, n in zip(entries, sizes):
        e.param, e.exp_avg, e.exp_avg_sq, e.numel = 0x1000, 0x3000, 0x4000, n
        if bits == 8:
            e.exp_avg_scale, e.exp_avg_sq_scale = 0x6000, 0x7000
    g = (ctypes.c_void_p * len(sizes))(*[0x2000 if x else None for x in grads])
    return _adamw._library().adamw_step(len(sizes), entries, g, 1, 0, bits, 1e-3, 0.9, 0.99, eps, 0.1, 1, None, None, None,
                                        0, None)


def test_the_limit_is_the_headers():
    text = open(os.path.join(ROOT, "include", "fp8q_adamw.h")).read()
    assert re.search(r"#define FP8Q_ADAMW_MAX_NUMEL \(\(1LL << 34\) - 1024\)", text)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("numel", [MOST + 1, 1 << 34, 1 << 39])
def test_a_tensor_past_a_launch(numel, bits):
    assert _step([numel], [True], bits) == ERR_SHAPE
    # behind as many others as fill more than one launch
    assert _step([0] * 130 + [numel], [True] * 131, bits) == ERR_SHAPE
    # (one that takes no part in the step may have any size)
    assert _step([MOST, numel], [False, False], bits) == OK


@pytest.mark.parametrize("eps,want", [(0.0, OK), (1e-8, OK), (1e-45, OK), (3.4e38, OK), (1e-46, ERR_SHAPE),
                                      (1e-50, ERR_SHAPE), (5e-324, ERR_SHAPE), (1e39, ERR_SHAPE), (1e308, ERR_SHAPE)])
def test_eps_is_what_float32_has_of_it(eps, want):
    """A positive eps that FP32 rounds to 0 would make elements without any gradient yet NaN (0 / 0)."""
    assert _step([0], [True], eps=eps) == want
