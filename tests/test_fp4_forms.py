"""The tests' sizes reach every form that the FP4 products' rules can choose, and
the tile kernels in every remainder of K: a change of the rules that takes a
form out of the tests shows here."""
from __future__ import annotations

import shutil

import pytest

import fp4_forms
import launch_rules

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

SIZES = sorted({s for p in range(0, 14) for s in (1 << p, (1 << p) + 1, (1 << p) * 5 // 4, (1 << p) * 3 // 2, (1 << p) * 7 // 4)})


def reachable_dense():
    return {launch_rules.gemm_form(m, n) for m in SIZES for n in SIZES}


def reachable_grouped():
    return {launch_rules.grouped_form(groups * rows, n, groups) for groups in (1, 2, 3, 4, 8, 16, 32, 64, 200)
            for rows in (0, 1, 8, 16, 20, 24, 32, 40, 48, 64, 100, 128, 256, 512, 2048) for n in SIZES}


def test_the_dense_sizes_reach_every_form():
    reached = {launch_rules.gemm_form(m, n) for m, n, _ in fp4_forms.DENSE}
    assert reachable_dense() == reached and len(reached) == 10


def test_the_grouped_sizes_reach_every_form():
    reached = {launch_rules.grouped_form(fp4_forms.m_total(c), c[1], len(c[0])) for c in fp4_forms.EXPERTS}
    assert reachable_grouped() == reached and len(reached) == 9


def rest(k):
    return -(-k // 128) % 4


def test_the_tile_kernels_see_every_remainder_of_k_and_ragged_edges():
    for size in (4, 8):
        cases = [c for c in fp4_forms.DENSE if launch_rules.gemm_form(*c[:2]) == ("tiles", size, size)]
        assert {rest(k) for _, _, k in cases} == {0, 1, 2, 3}
        assert any(m % 16 and n % 16 for m, n, _ in cases) and any(n % 8 == 0 and n % 128 for _, n, _ in cases)
    cases = [c for c in fp4_forms.EXPERTS
             if launch_rules.grouped_form(fp4_forms.m_total(c), c[1], len(c[0]))[0] == "grouped tiles"]
    assert {rest(c[2]) for c in cases} == {0, 1, 2, 3}
    rows = {r for c in cases for r in c[0]}
    assert {0, 1, 127, 128, 129, 256, 257, 513} <= rows
    assert any(c[1] % 16 for c in cases) and any(c[1] % 256 == 0 for c in cases) and any(c[4] > 256 for c in cases)


def test_fewer_rows_than_experts_take_the_narrow_pieces():
    for n in (1000, 4096, 8192):
        assert launch_rules.grouped_form(48, n, 70)[:2] == ("rows", 1)
