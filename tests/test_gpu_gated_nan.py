"""NaN and infinities in the gradients' E4M3 output: whatever else a tile holds,
it does not read back as a finite gradient; other tiles keep their bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fine_grained_fp8_quantize_amd as fq
from gpu_util import host_codes
from oracle import gated as model

pytestmark = pytest.mark.gpu

M, N = 256, 256
NAN, INF = float("nan"), float("inf")


def _inputs(seed):
    rng = np.random.default_rng(seed)
    dh = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).to(torch.bfloat16).cuda()
    gu = torch.from_numpy(rng.standard_normal((M, 2 * N)).astype(np.float32)).to(torch.bfloat16).cuda()
    return dh, gu


def _check(dh, gu, clean_dh, clean_gu, bad, act, transposed):
    """`bad`: [M][2N], elements of D that are not finite. Tiles with one read back as nothing finite."""
    got = fq.fp8_gated_backward(dh, gu, act, transposed=transposed)
    clean = fq.fp8_gated_backward(clean_dh, clean_gu, act, transposed=transposed)
    views = [(got[0], got[1], clean[0], clean[1], bad)]
    if transposed:
        views.append((got[2], got[3], clean[2], clean[3], bad.T))
    for q, s, cq, cs, b in views:
        q, s, cq, cs = host_codes(q), s.cpu().numpy(), host_codes(cq), cs.cpu().numpy()
        tile = np.repeat(b.reshape(b.shape[0], -1, 128).any(2), 128, 1)
        with np.errstate(invalid="ignore"):
            v = model.values(q, s, 1)
        assert not np.isfinite(v[tile]).any(), "tiles with one"
        assert np.array_equal(q[~tile], cq[~tile]), "codes of the others"
        t = tile[:, ::128].T
        assert np.array_equal(s[~t], cs[~t]), "scales of the others"


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("others", [1.0, 0.0, 2.0 ** -75])
def test_one_in_a_tile(value, others, transposed, act):
    """`others`: the factor of the rest of the gradient; 2^-75 gives scales below 2^-60."""
    dh, gu = _inputs(1)
    dh *= others
    gu[gu == 0] = 1.0  # (an infinity times zero is no infinity)
    clean, bad = dh.clone(), np.zeros((M, 2 * N), bool)
    for row, col in ((0, 0), (5, 131), (130, 77), (255, 255)):
        dh[row, col] = value
        bad[row, [col, col + N]] = True
    _check(dh, gu, clean, gu, bad, act, transposed)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("transposed", [False, True])
def test_rows_and_all_of_nan(transposed, act):
    dh, gu = _inputs(2)
    clean, bad = dh.clone(), np.zeros((M, 2 * N), bool)
    dh[[3, 140]] = NAN
    bad[[3, 140]] = True
    _check(dh, gu, clean, gu, bad, act, transposed)
    dh[:] = NAN
    bad[:] = True
    _check(dh, gu, clean, gu, bad, act, transposed)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_nan_in_gate_and_up(sign, transposed, act):
    """A gate's is both gradients', an up's the gate's alone; beside zeros, and of either sign."""
    dh, gu = _inputs(3)
    dh[:, 128:] = 0.0
    clean, bad = gu.clone(), np.zeros((M, 2 * N), bool)
    nan = torch.tensor([0x7FC0 if sign > 0 else -0x40], dtype=torch.int16, device="cuda").view(torch.bfloat16)
    gu[7, 200], gu[9, 5] = nan[0], nan[0]
    bad[7, [200, 200 + N]], bad[9, [5, 5 + N]] = True, True
    gu[201, N + 140] = nan[0]
    bad[201, 140] = True
    _check(dh, gu, dh, clean, bad, act, transposed)
