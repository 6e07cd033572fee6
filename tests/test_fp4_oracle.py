"""CPU pins of the FP4 oracle: the E2M1 grid by hand, ties, saturation, the
scale rule, non-finite blocks, and the tile layout by its formula."""
from __future__ import annotations

import numpy as np
import pytest

import workloads as wl
from oracle import fp4


@pytest.mark.parametrize("v,code", [
    (0.0, 0), (0.25, 0), (0.26, 1), (0.5, 1), (0.75, 2), (0.74, 1), (1.0, 2), (1.25, 2), (1.26, 3), (1.5, 3),
    (1.75, 4), (2.0, 4), (2.5, 4), (2.51, 5), (3.0, 5), (3.5, 6), (4.0, 6), (5.0, 6), (5.01, 7), (6.0, 7), (7.99, 7)])
def test_encode_by_hand(v, code):
    assert fp4.encode(np.array([v, -v])).tolist() == [code, code + 8]


def test_every_code_is_its_own_nearest():
    assert fp4.encode(fp4.VALUES).tolist() == list(range(16))


@pytest.mark.parametrize("amax,byte", [
    (6.0, 127), (4.0, 127), (7.96875, 127), (8.0, 128), (3.984375, 126), (1.0, 125), (2.0 ** -125, 0), (2.0 ** -124, 1),
    (2.0 ** -133, 0), (0.0, 0), (2.0 ** 127, 252)])
def test_scale_rule(amax, byte):
    x = np.zeros((1, 32), np.float32)
    x[0, 5] = amax
    _, e = fp4.quantize(wl.f32_to_bf16_bits(x))
    assert e.tolist() == [[byte]]


def test_non_finite_block_reads_back_as_nan_and_the_others_do_not():
    x = wl.f32_to_bf16_bits(np.ones((2, 96), np.float32))
    x[0, 40] = 0x7F80
    x[1, 95] = 0x7FC1
    codes, e = fp4.quantize(x)
    v = fp4.values(codes, e)
    want = np.ones((2, 96))
    want[0, 32:64] = np.nan
    want[1, 64:] = np.nan
    assert np.array_equal(v, want, equal_nan=True)


def test_tiles_place_every_code_and_byte():
    rng = np.random.default_rng(5)
    rows, k = 37, 672
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    e = rng.integers(0, 255, (rows, k // 32)).astype(np.uint8)
    q, s = fp4.tiles(codes, e)
    assert q.shape == (6, 3, 1024) and s.shape == (2, 3, 64, 4)
    for r, c in ((0, 0), (0, 1), (5, 33), (36, 671), (15, 127), (16, 128), (12, 640)):
        b, rr = c % 128 // 32, r % 16
        byte = q[c // 128, r // 16, rr * 64 + (b ^ (rr // 4)) * 16 + c % 32 // 2]
        assert (byte >> (4 * (c & 1))) & 15 == codes[r, c]
        assert s[c // 512, r // 16, 4 * rr + b, c // 128 % 4] == e[r, c // 32]
    # what lies past the matrix is zero
    assert q.astype(np.int64).sum() == sum(int(v) << (4 * (i % 2)) for row in codes for i, v in enumerate(row))
