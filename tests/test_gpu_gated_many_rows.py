"""Experts of millions of rows: every row of the gated products is written once,
with its own expert's weights, also where the split into tiles passes 32 bits."""
from __future__ import annotations

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _free():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("codes", [False, True])
def test_an_expert_of_six_million_rows(codes):
    """Rows of ones; an expert's weights are one column of a single value each, so all of its rows give one H."""
    rows, n, k = (256, 6000000, 256), 128, 128
    off = torch.tensor([0, 256, 6000256, 6000512], dtype=torch.int32, device="cuda")
    m = sum(rows)
    a = torch.full((m, k), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    a_s = torch.ones((1, m), device="cuda")
    b = torch.zeros((3, 2, n, k), dtype=torch.uint8, device="cuda")
    b[:, :, :, 5] = 0x38
    # gate and up are both 1, 2, 4: H = v silu(v)
    b_s = torch.tensor([1.0, 2.0, 4.0], device="cuda").reshape(3, 1, 1, 1).expand(3, 2, 1, 1).contiguous()
    v = torch.tensor([1.0, 2.0, 4.0], dtype=torch.float64)
    want = (v * v / (1 + torch.exp(-v))).tolist()
    # (few last places of FP32 in H, and bf16's rounding, or those of the scale and its product with 448)
    if codes:
        out = torch.full((m, n), 0x7F, dtype=torch.uint8, device="cuda")
        scale = torch.full((1, m), float("nan"), device="cuda")
        fq.fp8_grouped_gated_gemm(off, None, a, a_s, b, b_s, out_dtype=E4M3, out=out, scale=scale)
        assert bool((out == 0x7E).all())  # 448
        got, room = scale[0] * 448, 2.0 ** -20
    else:
        out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
        fq.fp8_grouped_gated_gemm(off, None, a, a_s, b, b_s, out=out)
        assert bool((out == out[:, :1]).all())
        got, room = out[:, 0].float(), 2.0 ** -8 * 1.001
    at = 0
    for r, x in zip(rows, want):
        part = got[at:at + r]
        assert abs(float(part[0]) - x) <= room * x and bool((part == part[0]).all()), (r, x)
        at += r
