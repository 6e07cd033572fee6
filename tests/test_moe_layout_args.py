"""moe_dispatch's plain numbers: what 32 bits do not hold is refused, not cut
to its low half."""
from __future__ import annotations

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from fine_grained_fp8_quantize_amd import _moe

# experts, align, first
BAD = [(0, 16, 0), (-5, 16, 0), (1025, 16, 0), ((1 << 32) + 8, 16, 0), (8, 0, 0), (8, -16, 0), (8, (1 << 32) + 16, 0),
       (8, 16, -1), (8, 16, 1 << 32), (8, 16, 0x7FFFFFFF - 7)]


@pytest.mark.parametrize("experts,align,first", BAD)
def test_refused(experts, align, first):
    with pytest.raises(fq.Fp8qError):
        _moe._layout_args(experts, align, first)


@pytest.mark.parametrize("experts,align,first", [(1, 1, 0), (1024, 128, 0), (8, 16, 0x7FFFFFFF - 8)])
def test_taken(experts, align, first):
    _moe._layout_args(experts, align, first)


@pytest.mark.gpu
def test_refused_by_the_call():
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for experts, align, first in BAD:
        with pytest.raises(fq.Fp8qError):
            fq.moe_dispatch(ids, experts, align, first)
    _, _, dst = fq.moe_dispatch(ids, 8, 16, 0x7FFFFFFF - 8)
    assert (dst == -1).all()
