"""What a row's weight-only product depends on: not on its place nor on what the
other rows hold, whatever their number; that number may pick another order of the
same FP32 sums, which then agree within their error bound."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _problem(m, n, k, lead=()):
    rng = np.random.default_rng(m + n)
    w = torch.from_numpy((rng.standard_normal((int(np.prod((1, *lead))), n, k)) * 0.05).astype(np.float32))
    q, s = fq.fp4_quantize_mx(w.to(torch.bfloat16).cuda())
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).to(torch.bfloat16).cuda()
    return rng, x, q.reshape(*lead, *q.shape[1:]), s.reshape(*lead, *s.shape[1:])


SHAPES = [(2, 2048, 7168), (16, 2048, 7168), (17, 2048, 7168), (64, 2048, 7168), (150, 300, 4100), (33, 5000, 1024)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("gated", [False, True])
def test_place_and_neighbours_do_not_matter(m, n, k, gated):
    rng, x, q, s = _problem(m, n, k, (2,) if gated else ())
    fn = (lambda t: fq.fp4_gated_gemv_mx(t, q, s, n, out_dtype=torch.float32)) if gated else (
        lambda t: fq.fp4_gemv_mx(t, q, s, n, out_dtype=torch.float32))
    want = fn(x)
    assert torch.equal(fn(x), want)
    order = torch.from_numpy(rng.permutation(m)).cuda()
    assert torch.equal(fn(x[order]), want[order])
    keep = m // 2
    for other in (float("nan"), float("inf"), 0.0, 1e30):
        y = torch.full_like(x, other)
        y[keep] = x[keep]
        assert torch.equal(fn(y)[keep], want[keep]), other


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_numbers_of_rows_agree_within_the_sums_bound(m, n, k):
    _, x, q, s = _problem(m, n, k)
    v = fq.fp4_dequantize_mx(q, s, n, k, torch.float32).double()
    for i in (0, m - 1):
        row = x[i:i + 1]
        one, all_ = (fq.fp4_gemv_mx(t, q, s, n, out_dtype=torch.float32).double()[j] for t, j in ((row, 0), (x, i)))
        # either sum of K exact products is off by at most K U times the sum of magnitudes
        room = 2 * 1.01 * k * U * (row.double().abs() @ v.abs().t().contiguous())[0]
        assert bool(((one - all_).abs() <= room).all())


def test_routes_of_an_expert_in_any_order():
    rng, x, q, s = _problem(40, 96, 2000, (3,))
    ids = torch.from_numpy(rng.integers(-1, 4, (40, 2)).astype(np.int32)).cuda()
    want = fq.fp4_gemv_mx(x, q, s, 96, ids, out_dtype=torch.float32)
    order = torch.from_numpy(rng.permutation(40)).cuda()
    got = fq.fp4_gemv_mx(x[order], q, s, 96, ids[order].contiguous(), out_dtype=torch.float32)
    assert torch.equal(got, want[order])
    y = torch.full_like(x, float("nan"))
    y[7] = x[7]
    assert torch.equal(fq.fp4_gemv_mx(y, q, s, 96, ids, out_dtype=torch.float32)[7], want[7])
