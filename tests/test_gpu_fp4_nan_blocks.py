"""A scale byte of 255 is NaN whatever codes stand under it (a matrix that did not
come from this library's quantizers): read back, and in products by either
operand, few rows and many."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from oracle import fp4

pytestmark = pytest.mark.gpu


def matrix(seed, rows, k):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    return codes, rng.integers(120, 132, (rows, k // 32)).astype(np.uint8)


def on_gpu(codes, ebytes):
    q, s = fp4.tiles(codes, ebytes)
    return torch.from_numpy(q).cuda(), torch.from_numpy(s.view(np.int32).reshape(s.shape[:3])).cuda()


def test_read_back():
    codes, e = matrix(1, 40, 640)
    e[7, 3] = e[39, 19] = e[0, 0] = 255
    codes[7, 96:112] = np.arange(16)  # every code under one of them
    want = fp4.values(codes, e)
    for dt in (torch.bfloat16, torch.float32):
        got = fq.fp4_dequantize_mx(*on_gpu(codes, e), 40, 640, dt).double().cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("m,n", [(3, 40), (40, 300), (700, 2050), (4000, 4000)])
def test_products(m, n):
    k = 640
    (ac, ae), (bc, be) = matrix(2, m, k), matrix(3, n, k)
    ae[m - 1, 5], be[n - 2, 11], be[0, 0] = 255, 255, 255
    c = torch.isnan(fq.fp4_gemm_mx(*on_gpu(ac, ae), *on_gpu(bc, be), m, n, torch.float32)).cpu().numpy()
    want = np.zeros((m, n), bool)
    want[m - 1], want[:, n - 2], want[:, 0] = True, True, True
    assert np.array_equal(c, want)
