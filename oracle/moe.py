"""CPU oracle for the MoE routing operators: the expert-sorted row layout by a
walk over the routes, the balance loss and its gradient from their formulas in
float64. TEST INFRASTRUCTURE ONLY, as the rest of ``oracle``."""
from __future__ import annotations

import numpy as np


def dispatch(ids: np.ndarray, experts: int, align: int, first: int):
    """(group_offsets, group_rows, dst_rows) as int64 arrays."""
    rows = np.zeros(experts, np.int64)
    place = np.full(ids.shape, -1, np.int64)
    for t in range(ids.shape[0]):
        for k in range(ids.shape[1]):
            e = int(ids[t, k]) - first
            if 0 <= e < experts:
                place[t, k] = rows[e]
                rows[e] += 1
    off = np.zeros(experts + 1, np.int64)
    for e in range(experts):
        off[e + 1] = off[e] + -(-rows[e] // align) * align
    local = np.clip(ids.astype(np.int64) - first, 0, experts - 1)
    return off, rows, np.where(place >= 0, off[local] + place, -1)


def scores(x: np.ndarray, score: str) -> np.ndarray:
    """Row scores in float64; rows without a finite score are zero. Both kinds
    as a softmax: of the logits, or of their log sigmoids."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        u = x if score == "softmax" else -np.logaddexp(0.0, -x)
        top = u.max(axis=1, keepdims=True)
        e = np.exp(u - np.where(np.isneginf(top), 0.0, top))
        s = e.sum(axis=1, keepdims=True)
        return np.where(s == 0, 0.0, e / np.where(s == 0, 1.0, s))


def balance(x: np.ndarray, ids: np.ndarray, offsets, score: str, alpha: float):
    """(loss, counts [S][E], coef [S][E])."""
    experts, seqs = x.shape[1], len(offsets) - 1
    valid = (ids >= 0) & (ids < experts)
    counts, coef = np.zeros((seqs, experts), np.int64), np.zeros((seqs, experts))
    p, losses = scores(x, score), []
    for s in range(seqs):
        rows = [t for t in range(offsets[s], offsets[s + 1]) if valid[t].any()]
        for t in rows:
            for e in ids[t][valid[t]]:
                counts[s, e] += 1
        if rows:
            f = experts * counts[s] / counts[s].sum()
            losses.append(alpha * float((f * p[rows].mean(axis=0)).sum()))
            coef[s] = alpha * f / len(rows)
    n = max(1, len(losses))
    return sum(losses) / n, counts, coef / n


def balance_gradient(x: np.ndarray, ids: np.ndarray, offsets, score: str, coef: np.ndarray, grad: float) -> np.ndarray:
    experts = x.shape[1]
    p, out = scores(x, score), np.zeros_like(x)
    for s in range(len(offsets) - 1):
        for t in range(offsets[s], offsets[s + 1]):
            if ((ids[t] >= 0) & (ids[t] < experts)).any():
                d = grad * p[t] * (coef[s] - (p[t] * coef[s]).sum())
                if score == "sigmoid":
                    with np.errstate(over="ignore"):
                        d = d / (1.0 + np.exp(x[t]))
                out[t] = d
    return out
