"""FP4 matrices of more than 2^32 bytes of codes: the ends of the arrays against
the same operators on their last rows alone. The values are small integers, so
every sum is exact in FP32 and the comparisons are bit for bit."""
from __future__ import annotations

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq

pytestmark = pytest.mark.gpu

ROWS, K, LAST = 70000, 131072, 32


@pytest.fixture(scope="module")
def big():
    torch.manual_seed(0)
    x = torch.randint(-1, 3, (ROWS, K), dtype=torch.int8, device="cuda").bfloat16()
    yield x
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tiling", ["1x32", "32x1"])
def test_quantize_read_back_and_multiply(big, tiling):
    x = big if tiling == "1x32" else big.view(K, ROWS)
    tail = x[-LAST:] if tiling == "1x32" else x[:, -LAST:]
    q, s = fq.fp4_quantize_mx(x, tiling)
    assert q.numel() > 1 << 32
    q1, s1 = fq.fp4_quantize_mx(tail.contiguous(), tiling)
    assert torch.equal(q[:, -LAST // 16:], q1) and torch.equal(s[:, -LAST // 16:], s1)
    for m in (1, 40, 300):
        a = fq.fp4_quantize_mx(torch.randint(-1, 2, (m, K), dtype=torch.int8, device="cuda").bfloat16())
        c = fq.fp4_gemm_mx(*a, q, s, m, ROWS, torch.float32)
        assert torch.equal(c[:, -LAST:], fq.fp4_gemm_mx(*a, q1, s1, m, LAST, torch.float32))
        # and as the row operand
        c = fq.fp4_gemm_mx(q, s, *a, ROWS, m, torch.float32)
        assert torch.equal(c[-LAST:], fq.fp4_gemm_mx(q1, s1, *a, LAST, m, torch.float32))
    y = fq.fp4_dequantize_mx(q, s, ROWS, K)
    assert torch.equal(y[-LAST:], tail if tiling == "1x32" else tail.t())


def test_experts_past_the_edge(big):
    """Experts' weights whose last one starts past 2^32 bytes."""
    experts, n, k = 70, 1000, K
    w = fq.fp4_quantize_mx(big.view(experts, n, k))
    assert (experts - 1) * w[0][0].numel() > 1 << 32
    rows = torch.zeros(experts, dtype=torch.int32, device="cuda")
    rows[-1], rows[0] = 5, 20
    off = torch.tensor([0] + [32] * (experts - 1) + [48], dtype=torch.int32, device="cuda")
    x = torch.randint(-1, 2, (48, k), dtype=torch.int8, device="cuda").bfloat16()
    c = fq.fp4_grouped_gemm_mx(off, rows, *fq.fp4_quantize_mx(x), *w, n, torch.float32)
    for beg, count, e in ((0, 20, 0), (32, 5, experts - 1)):
        one = fq.fp4_gemm_mx(*fq.fp4_quantize_mx(x[beg:beg + count]), w[0][e], w[1][e], count, n, torch.float32)
        assert torch.equal(c[beg:beg + count], one)
    assert (c[20:32] == 0).all() and (c[37:] == 0).all()
