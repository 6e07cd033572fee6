"""GPU parity of every form of the FP4 products' kernels against float64.

The operands are the values that the matrices hold (``fp4_dequantize_mx``, which
other tests hold to the oracle bit for bit). An output is a sum of tile products
in FP32: it is off by at most one FP32 rounding of the running sum (at most
sum |a||b|) per K tile of 128 and per joined partial (16 at the most), doubled
for the adds inside the matrix core; bf16 output adds half a unit of 8
significant bits."""
from __future__ import annotations

import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
import fp4_forms
from gpu_util import nan_out

pytestmark = pytest.mark.gpu

OUT = [torch.bfloat16, torch.float32]


def act(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    big = torch.rand(shape, generator=g, device="cuda") < 1e-3
    return torch.where(big, x * 50, x).bfloat16()


def values(q, s, rows, k):
    return fq.fp4_dequantize_mx(q, s, rows, k, torch.float32).double()


def check(got, a, b, out_dtype, what):
    ref = a @ b.t()
    tol = (-(-a.shape[1] // 128) + 16) * 2.0 ** -23 * (a.abs() @ b.abs().t())
    if out_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    bad = ~((got.double() - ref).abs() <= tol + 1e-300)
    assert not bad.any(), "%s: %d outputs off, or not written" % (what, int(bad.sum()))


@pytest.mark.parametrize("m,n,k", fp4_forms.DENSE)
@pytest.mark.parametrize("out_dtype", OUT)
def test_dense(m, n, k, out_dtype):
    print(m, n, k, flush=True)
    a, sa = fq.fp4_quantize_mx(act(1, m, k))
    b, sb = fq.fp4_quantize_mx((act(2, n, k).float() * 0.02).bfloat16())
    # rows of C in a wider array: nothing outside them is written
    wide = torch.full((m, n + 8), 3.0, dtype=out_dtype, device="cuda")
    wide[:, :n] = float("nan")
    fq.fp4_gemm_mx(a, sa, b, sb, m, n, out_dtype, out=wide[:, :n])
    check(wide[:, :n], values(a, sa, m, k), values(b, sb, n, k), out_dtype, "%d x %d x %d" % (m, n, k))
    assert (wide[:, n:] == 3).all(), "written outside the output"
    if n % 8:  # and with rows that start on 16-byte boundaries or do not, the other way round
        out = fq.fp4_gemm_mx(a, sa, b, sb, m, n, out_dtype, out=nan_out((m, n), out_dtype))
        assert torch.equal(out, wide[:, :n])


@pytest.mark.parametrize("case", fp4_forms.EXPERTS, ids=lambda c: "%dx%d-%dx%d" % (len(c[0]), max(c[0]), c[1], c[2]))
@pytest.mark.parametrize("out_dtype", OUT)
def test_experts(case, out_dtype):
    rows, n, k, align, extra = case
    print(case, flush=True)
    m_total, segments = fp4_forms.m_total(case), fp4_forms.padded(rows, align)
    beg = [sum(segments[:e]) for e in range(len(rows) + 1)]
    x, real = act(3, m_total, k), torch.zeros(m_total, dtype=torch.bool, device="cuda")
    for e, r in enumerate(rows):
        real[beg[e]:beg[e] + r] = True
    clean = fq.fp4_quantize_mx(x)
    x[~real, 0] = float("nan")  # padding rows may hold anything
    a, sa = fq.fp4_quantize_mx(x)
    b, sb = fq.fp4_quantize_mx((act(4, len(rows), n, k).float() * 0.02).bfloat16())
    off = torch.tensor(beg, dtype=torch.int32, device="cuda")
    counts = torch.tensor(rows, dtype=torch.int32, device="cuda")
    ldc = -(-n // 8) * 8 + 8
    wide = torch.full((m_total, ldc), 3.0, dtype=out_dtype, device="cuda")
    wide[:, :n] = float("nan")
    c = fq.fp4_grouped_gemm_mx(off, counts, a, sa, b, sb, n, out_dtype, out=wide[:, :n])
    av = values(*clean, m_total, k)
    for e, r in enumerate(rows):
        if r:
            check(c[beg[e]:beg[e] + r], av[beg[e]:beg[e] + r], values(b[e], sb[e], n, k), out_dtype, "expert %d" % e)
    assert (c[~real] == 0).all(), "padding rows not zero"
    assert (wide[:, n:] == 3).all(), "written outside the output"


def test_experts_of_the_tile_kernel_past_the_edge():
    """Weights of 40 experts, the last of which starts past 2^32 bytes of codes.
    The values are small integers, so every sum is exact in FP32 and the
    comparison is bit for bit."""
    experts, n, k = 40, 2048, 131072
    q = torch.empty((experts, k // 128, n // 16, 1024), dtype=torch.uint8, device="cuda")
    s = torch.empty((experts, k // 512, n // 16, 64), dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    for e in range(experts):
        w = torch.randint(-1, 3, (n, k), generator=g, dtype=torch.int8, device="cuda").bfloat16()
        fq.fp4_quantize_mx(w, q=q[e], scale=s[e])
    assert (experts - 1) * q[0].numel() > 1 << 32
    rows = [20] + [0] * (experts - 3) + [1, 300]
    segments = fp4_forms.padded(rows, 16)
    beg = [sum(segments[:e]) for e in range(experts + 1)]
    m_total = beg[-1] + 400
    assert m_total >= experts
    x = torch.randint(-1, 2, (m_total, k), generator=g, dtype=torch.int8, device="cuda").bfloat16()
    a, sa = fq.fp4_quantize_mx(x)
    c = fq.fp4_grouped_gemm_mx(torch.tensor(beg, dtype=torch.int32, device="cuda"),
                               torch.tensor(rows, dtype=torch.int32, device="cuda"), a, sa, q, s, n, torch.float32,
                               out=nan_out((m_total, n), torch.float32))
    for e in (0, experts - 2, experts - 1):
        lo, hi = beg[e], beg[e] + rows[e]
        one = fq.fp4_gemm_mx(*fq.fp4_quantize_mx(x[lo:hi]), q[e], s[e], rows[e], n, torch.float32)
        assert torch.equal(c[lo:hi], one), e
        assert (c[hi:beg[e + 1]] == 0).all()
    assert (c[beg[-1]:] == 0).all()
