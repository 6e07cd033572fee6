"""The grouped FP4 product of a rank that holds no expert: every row lies past
the last segment, so the output is zeros."""
from __future__ import annotations

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from gpu_util import nan_out

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [None, torch.empty(0, dtype=torch.int32)])
def test_no_experts_give_zeros(rows):
    m, n, k = 48, 40, 256
    a, sa = fq.fp4_quantize_mx(torch.ones((m, k), dtype=torch.bfloat16, device="cuda"))
    b, sb = fq.fp4_quantize_mx(torch.empty((0, n, k), dtype=torch.bfloat16, device="cuda"))
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = None if rows is None else rows.cuda()
    for dt in (torch.bfloat16, torch.float32):
        wide = nan_out((m, n + 8), dt)
        c = fq.fp4_grouped_gemm_mx(off, rows, a, sa, b, sb, n, dt, out=wide[:, :n])
        assert (c == 0).all() and torch.isnan(wide[:, n:]).all()
    side = torch.cuda.Stream()
    out = nan_out((m, n), torch.bfloat16)
    torch.cuda.synchronize()
    c = fq.fp4_grouped_gemm_mx(off, rows, a, sa, b, sb, n, out=out, stream=side)
    side.synchronize()
    assert (c == 0).all()
