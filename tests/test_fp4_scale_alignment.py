"""FP4 products whose scales are aligned to their words only. The tile kernels
copy scales 16 bytes at a time, so such scales must not reach them; the results
are the aligned scales' own, bit for bit, on sums that are exact in FP32."""
from __future__ import annotations

import shutil

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
import launch_rules

DENSE = [(600, 1500, 640), (700, 2048, 640), (4096, 4096, 1024)]         # m, n, k
EXPERTS = [([300, 5, 0, 128, 257, 40], 4096, 640), ([33] * 40, 2300, 1664)]  # rows, n, k


def padded(rows):
    return sum(-(-r // 16) * 16 for r in rows)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_the_tile_kernels_take_aligned_scales_only():
    for m, n, _ in DENSE:
        assert launch_rules.gemm_form(m, n)[0] == "tiles"
        assert launch_rules.gemm_form(m, n, False)[0] == "rows"
    for rows, n, _ in EXPERTS:
        assert launch_rules.grouped_form(padded(rows), n, len(rows))[0] == "grouped tiles"
        assert launch_rules.grouped_form(padded(rows), n, len(rows), False)[0] == "rows"
    # where scales do not matter, they do not matter
    for m, n in ((1, 4096), (20, 4096), (64, 2048)):
        assert launch_rules.gemm_form(m, n) == launch_rules.gemm_form(m, n, False)


def shifted(s, words):
    """The same words ``words`` * 4 bytes off a 16-byte boundary."""
    buf = torch.empty(s.numel() + words + 4, dtype=torch.int32, device="cuda")
    assert buf.data_ptr() % 16 == 0
    out = buf[words:words + s.numel()].view(s.shape)
    out.copy_(s)
    return out


def integers(seed, *shape):
    """Small integers, exact in FP4: the sums are exact in FP32, in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", DENSE)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_dense(m, n, k, out_dtype):
    a, sa = fq.fp4_quantize_mx(integers(1, m, k))
    b, sb = fq.fp4_quantize_mx(integers(2, n, k))
    want = fq.fp4_gemm_mx(a, sa, b, sb, m, n, out_dtype)
    for da, db in ((1, 0), (0, 2), (3, 1)):
        got = fq.fp4_gemm_mx(a, shifted(sa, da), b, shifted(sb, db), m, n, out_dtype)
        assert torch.equal(got, want), (da, db)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k", EXPERTS)
def test_experts(rows, n, k):
    off = torch.tensor([0] + [padded(rows[:i + 1]) for i in range(len(rows))], dtype=torch.int32, device="cuda")
    counts = torch.tensor(rows, dtype=torch.int32, device="cuda")
    m_total = padded(rows)
    a, sa = fq.fp4_quantize_mx(integers(3, m_total, k))
    b, sb = fq.fp4_quantize_mx(integers(4, len(rows), n, k))
    want = fq.fp4_grouped_gemm_mx(off, counts, a, sa, b, sb, n, torch.float32)
    # arrays that start off a boundary, and experts an odd number of words apart
    got = fq.fp4_grouped_gemm_mx(off, counts, a, shifted(sa, 1), b, shifted(sb, 3), n, torch.float32)
    assert torch.equal(got, want)
    per = sb[0].numel()
    buf = torch.zeros(len(rows) * (per + 1) + 4, dtype=torch.int32, device="cuda")
    odd = buf[:len(rows) * (per + 1)].view(len(rows), per + 1)[:, :per].view(sb.shape)
    odd.copy_(sb)
    got = fq.fp4_grouped_gemm_mx(off, counts, a, sa, b, odd, n, torch.float32)
    assert odd.stride(0) == per + 1 and torch.equal(got, want)


@pytest.mark.gpu
def test_the_values_themselves():
    """Against the product of the values that the operands hold."""
    m, n, k = 600, 1500, 640
    a, sa = fq.fp4_quantize_mx(integers(5, m, k))
    b, sb = fq.fp4_quantize_mx(integers(6, n, k))
    av, bv = fq.fp4_dequantize_mx(a, sa, m, k, torch.float32), fq.fp4_dequantize_mx(b, sb, n, k, torch.float32)
    want = (av.double().cpu() @ bv.double().cpu().t()).float()
    got = fq.fp4_gemm_mx(a, shifted(sa, 1), b, shifted(sb, 1), m, n, torch.float32)
    assert torch.equal(got.cpu(), want)
