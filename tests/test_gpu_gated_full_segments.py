"""Experts whose rows are all real, without group_rows: on either side of the rule
that sends them to tiles, against the float64 oracle and the counted call."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from gpu_util import host_codes
from oracle import gated as model
from test_gpu_gated import E4M3, _close, _dev, _finite, _problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,n,k", [((128, 0, 256, 128), 512, 384), ((128,) * 4, 1024, 256), ((128,) * 4, 1160, 256),
                                      ((512,), 2048, 512), ((128,) * 8, 640, 384), ((256, 128), 200, 128)])
def test_all_rows_real(rows, n, k):
    off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    m = int(off[-1])
    a, a_s, b, b_s = _problem(m + n, m, n, k, (len(rows),))
    want, gate, up = (np.zeros((m, n)) for _ in range(3))
    for e in range(len(rows)):
        at = slice(off[e], off[e + 1])
        if rows[e]:
            want[at], gate[at], up[at] = model.block("silu", a[at], a_s[:, at], b[e], b_s[e])
    d, counts = _dev(off, a, a_s, b, b_s), torch.tensor(rows, dtype=torch.int32, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        keep = torch.full((m, 2 * n), float("nan"), dtype=torch.bfloat16, device="cuda")
        out = torch.full((m, n), float("nan"), dtype=dt, device="cuda")
        fq.fp8_grouped_gated_gemm(d[0], None, *d[1:], "silu", dt, out=out, gate_up=keep)
        for got, ref, what in ((out, want, "H"), (keep[:, :n], gate, "gate"), (keep[:, n:], up, "up")):
            _close(_finite(got), ref, what)
        # (the counted call may take the other kernel: other orders of the same sums)
        _close(_finite(fq.fp8_grouped_gated_gemm(d[0], counts, *d[1:], "silu", dt)), want, "with counts")
    if n % 128 == 0:
        q, s = fq.fp8_grouped_gated_gemm(d[0], None, *d[1:], "silu", E4M3)
        want_q, want_s = model.tiles_1x128(_finite(out).astype(np.float32))
        assert np.array_equal(host_codes(q), want_q) and np.array_equal(s.cpu().numpy(), want_s)
