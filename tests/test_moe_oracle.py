"""CPU pins of the MoE oracle: a layout by hand, a loss by hand, the gradient
against central differences of the loss."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import moe


def test_dispatch_by_hand():
    ids = np.array([[3, 1], [1, -1], [2, 1], [9, 3]])
    off, rows, dst = moe.dispatch(ids, 3, 4, 1)          # experts 1..3
    assert rows.tolist() == [3, 1, 2]
    assert off.tolist() == [0, 4, 8, 12]
    assert dst.tolist() == [[8, 0], [1, -1], [4, 2], [-1, 9]]


def test_loss_by_hand():
    x = np.log(np.array([[1.0, 3.0], [1.0, 1.0], [2.0, 6.0]]))
    ids = np.array([[1], [0], [1]])
    loss, counts, coef = moe.balance(x, ids, [0, 2, 3], "softmax", 2.0)
    assert counts.tolist() == [[1, 1], [0, 1]]
    # f = (1, 1), P = (3/8, 5/8): 2 * 1; f = (0, 2), P = (1/4, 3/4): 2 * 1.5; mean
    assert loss == pytest.approx(2.5)
    assert coef == pytest.approx(np.array([[0.5, 0.5], [0.0, 2.0]]))


def test_rows_without_a_score_and_uncounted_rows():
    x = np.array([[-np.inf, -np.inf], [0.0, -np.inf], [5.0, 1.0]])
    ids = np.array([[0], [0], [-1]])
    for score in ("softmax", "sigmoid"):
        loss, counts, _ = moe.balance(x, ids, [0, 3], score, 1.0)
        assert counts.tolist() == [[2, 0]] and loss == pytest.approx(2 * 0.5)
    assert moe.balance(x, np.full((3, 1), -1), [0, 3], "softmax", 1.0)[0] == 0.0


def test_sigmoid_scores_are_normalised_sigmoids():
    x = np.random.default_rng(0).standard_normal((5, 7))
    s = 1 / (1 + np.exp(-x))
    assert moe.scores(x, "sigmoid") == pytest.approx(s / s.sum(1, keepdims=True))
    assert np.isfinite(moe.scores(x - 3000.0, "sigmoid")).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    rng = np.random.default_rng(1)
    x, ids, off = rng.standard_normal((9, 6)), rng.integers(-1, 6, (9, 2)), [0, 4, 4, 9]
    ids[2] = -1
    _, _, coef = moe.balance(x, ids, off, score, 0.7)
    g = moe.balance_gradient(x, ids, off, score, coef, 1.5)
    h = 1e-5
    for t in range(9):
        for e in range(6):
            hi, lo = x.copy(), x.copy()
            hi[t, e] += h
            lo[t, e] -= h
            d = (moe.balance(hi, ids, off, score, 0.7)[0] - moe.balance(lo, ids, off, score, 0.7)[0]) / (2 * h)
            assert g[t, e] == pytest.approx(1.5 * d, abs=1e-9)
