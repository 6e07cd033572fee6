"""The gradients' E4M3 codes and scales by the library's contract, bit for bit:
scales fl32(amax / 448), codes E4M3(fl32(x / s)). The gates are so large that the
logistic is 1, so a gradient is one product of two bf16 values and exact in FP32;
the products are those whose quotient lies next to the border of two codes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from gpu_util import assert_bits_equal, host_codes
from oracle import gated as model

pytestmark = pytest.mark.gpu

M, N = 256, 128


def _tiles(rng):
    """dh and g [M][N], all of their products exact: a row's first is its largest; of the rest, half are those whose
    code changes when the quotient is replaced by a product with the rounded reciprocal."""
    f = np.arange(128, 256)  # significands of bf16
    x = f[:, None] * f[None, :] / np.float32(4)  # g: 32 to 63.75
    rows = []
    while len(rows) < M:
        a, b = rng.integers(128, 256, 2)
        if a * b < 1 << 15:  # the largest of a row is 2^14 and more, the others are below
            continue
        s = np.float32(a * b / 2) / np.float32(448)
        y = (x / s).astype(np.float32)
        # (only quotients within a few last places of the middle of two codes can change)
        mant = y.view(np.int32) & 0xFFFFF
        near = np.argwhere(np.abs(mant - 0x80000) <= 4)
        near = near[[model.encode_e4m3(y[i, j, None])[0] != model.encode_e4m3((x[i, j, None] * (np.float32(1) / s)))[0]
                     for i, j in near]] if len(near) else near
        if len(near) == 0:
            continue
        pick = rng.integers(0, 128, (N, 2))
        pick[::2] = near[rng.integers(0, len(near), N // 2)]
        dh, g = f[pick[:, 0]].astype(np.float32), (f[pick[:, 1]] / 4.0).astype(np.float32)
        dh[0], g[0] = a, b / 2.0
        rows.append((dh * rng.choice([-1.0, 1.0], N).astype(np.float32), g))
    dh, g = np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])
    dh[5, 1], dh[6, 1] = 0.0, -0.0
    dh[7], dh[8] = 0.0, -0.0
    return dh, g


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("power", [0, -20, -85, -125, -133])
def test_codes_and_scales(power, transposed, act):
    """Powers whose scales are ordinary, below 2^-60, and (2^-133) subnormal."""
    dh, g = _tiles(np.random.default_rng(1))
    dh = np.ldexp(dh, power).astype(np.float32)
    x = dh * g
    if transposed:  # the searched tiles along the columns as well
        dh, g = np.concatenate((dh[:128], dh[128:].T)), np.concatenate((g[:128], g[128:].T))
        x = dh * g
    assert np.array_equal(x.astype(np.float64), dh.astype(np.float64) * g)
    d = torch.from_numpy(dh).to(torch.bfloat16).cuda()
    gate = torch.from_numpy(g).to(torch.bfloat16).cuda()
    out = fq.fp8_gated_backward(d, torch.cat((gate, gate), 1), act, transposed=transposed)
    both = np.concatenate((x, x), 1)  # dG = dH U act'(G) and dU = dH act(G), with U = G, act'(G) = 1, act(G) = G
    for q, s, ref in ((out[0], out[1], both), *(((out[2], out[3], both.T.copy()),) if transposed else ())):
        want_q, want_s = model.tiles_1x128(ref)
        assert_bits_equal(s.cpu().numpy(), want_s, "scales")
        assert_bits_equal(host_codes(q), want_q, "codes")
