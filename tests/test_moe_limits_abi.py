"""CPU checks of how large a batch the balance entry points take: past their
limits the host refuses the call before any launch."""
from __future__ import annotations

import os

import pytest

import fine_grained_fp8_quantize_amd as fq
from fine_grained_fp8_quantize_amd import _moe

ERR_SHAPE = 2
A, B, C, D, W = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


def _lib():
    if not os.path.exists(fq.library_path()):
        from fine_grained_fp8_quantize_amd import build
        build.build(force=False)
    return _moe._library()


def _forward(tokens, topk):
    return _lib().moe_balance_loss(A, 0, tokens, 8, 8, B, topk, C, 3, 0, 1.0, D, D, D, W, 1 << 40, None)


def _backward(tokens, topk):
    return _lib().moe_balance_loss_backward(A, 0, tokens, 8, 8, B, topk, C, 3, 0, D, D, W, 8, None)


@pytest.mark.parametrize("tokens,topk", [(1 << 28, 8), (1 << 30, 2), ((1 << 31) - 1, 8), ((1 << 31) // 3 + 1, 3)])
@pytest.mark.parametrize("call", [_forward, _backward])
def test_routes_that_an_int32_count_cannot_hold_are_refused(call, tokens, topk):
    assert tokens * topk > 0x7FFFFFFF
    assert call(tokens, topk) == ERR_SHAPE
