"""Launches stay within what a dispatch packet holds: fewer than 2^32
work-items in a grid. The sizes come from the headers that the launchers use."""
from __future__ import annotations

import shutil

import pytest

import launch_rules
from fine_grained_fp8_quantize_amd import _mx4

ERR_SHAPE = 2
X, Q, S, Y, D = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


def test_what_fits():
    fits = launch_rules.lib().launch_fits
    assert fits(0, 256) and fits((1 << 24) - 1, 256) and fits((1 << 31) - 1, 1)
    assert not fits(1 << 24, 256) and not fits(1 << 31, 1) and not fits(-1, 64)


def test_balance_gradient_of_the_longest_batch():
    tokens, piece = (1 << 31) - 1, launch_rules.lib().moe_backward_tokens()
    assert piece % 16 == 0
    for n in (1, 16, 17, piece, tokens % piece):
        blocks, threads = launch_rules.shape("moe_backward_shape", n)
        assert blocks == -(-n // 16) and launch_rules.lib().launch_fits(blocks, threads)
    # one launch for the whole batch would not fit
    blocks, threads = launch_rules.shape("moe_backward_shape", tokens)
    assert not launch_rules.lib().launch_fits(blocks, threads)


def fits(name, *args):
    return bool(launch_rules.lib().launch_fits(*launch_rules.shape(name, *args)))


def test_fp4_launch_sizes():
    # 16 rows x 512 k a wave, four waves a workgroup; 256 rows x 128 columns a workgroup of 512
    assert launch_rules.shape("fp4_quant_rows_shape", 2, 17, 513) == (2, 256)
    assert launch_rules.shape("fp4_quant_cols_shape", 1, 600, 130) == (8, 512)
    for name, rows in (("fp4_quant_rows_shape", 1 << 30), ("fp4_quant_cols_shape", 1 << 31)):
        assert fits(name, 1, rows - 4096, 8) and not fits(name, 1, rows, 8), name
    # the same number of 16 x 512 units: a transposing workgroup takes half of one where columns are few
    assert fits("fp4_quant_rows_shape", 1, 16, 1 << 31) and not fits("fp4_quant_cols_shape", 1, 1 << 31, 16)
    assert fits("fp4_gemm_shape", 16, 1 << 27, 64) and not fits("fp4_gemm_shape", 16, 1 << 28, 64)
    assert fits("fp4_gemm_shape", 4096, 4096, 56) and fits("fp4_grouped_shape", 8192, 4096, 56, 32)


# (only calls that the host refuses: a launch would read these addresses)
def test_fp4_calls_past_a_launch_are_refused():
    L = _mx4._library()
    big = 1 << 40
    assert L.fp4_quantize_mx(1, X, 1 << 30, 8, 8, 0, 0, Q, 1 << 26, 0, S, 1 << 26, 0, None) == ERR_SHAPE
    assert L.fp4_quantize_mx(1, X, 1 << 31, 8, 8, 0, 1, Q, 1, 0, S, 1, 0, None) == ERR_SHAPE
    assert L.fp4_quantize_mx(1 << 20, X, 1 << 14, 8, 8, 0, 0, Q, 1 << 10, big >> 10, S, 1 << 10, big >> 14, None) == ERR_SHAPE
    assert L.fp4_quantize_mx_scatter(X, 1 << 30, 8, 8, 1, D, 64, Q, 4, S, 4, None) == ERR_SHAPE
    assert L.fp4_dequantize_mx(Q, 1 << 26, S, 1 << 26, 1 << 30, 8, Y, 8, 0, None) == ERR_SHAPE
    n = 1 << 28
    assert L.fp4_gemm_mx(16, n, 8192, X, 1, S, 1, Q, n // 16, S, n // 16, Y, n, 0, None) == ERR_SHAPE
