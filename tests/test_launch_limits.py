"""Launches stay within what a dispatch packet holds: fewer than 2^32
work-items in a grid. The sizes come from the headers that the launchers use."""
from __future__ import annotations

import shutil

import pytest

import launch_rules

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
