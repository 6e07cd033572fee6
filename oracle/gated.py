"""CPU oracle of the gated feed-forward operators: activations and their slopes,
the block's products and gradients in float64, E4M3 tiles of float32 values.
TEST INFRASTRUCTURE ONLY, as the rest of ``oracle``."""
from __future__ import annotations

import numpy as np

from .adamw import decode_e4m3

_C = np.sqrt(2.0 / np.pi)


def _share(name: str, g: np.ndarray) -> np.ndarray:
    """act(g) / g: sigmoid(g), or (1 + tanh z) / 2 = sigmoid(2 z), which unlike 1 + tanh z does not cancel for z < 0."""
    w = g if name == "silu" else 2.0 * _C * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-w))


def act(name: str, g: np.ndarray) -> np.ndarray:
    g = np.asarray(g, np.float64)
    return g * _share(name, g)


def slope(name: str, g: np.ndarray) -> np.ndarray:
    g = np.asarray(g, np.float64)
    s = _share(name, g)
    by = 1.0 if name == "silu" else 2.0 * _C * (1.0 + 0.134145 * g * g)
    return s + g * s * (1.0 - s) * by


def values(q: np.ndarray, scale: np.ndarray, rows: int) -> np.ndarray:
    """float64 values of codes [r][k]: scale [k/128][r] (rows = 1) or [ceil(r/rows)][k/128]."""
    r, k = q.shape
    s = scale.T.astype(np.float64) if rows == 1 else np.repeat(scale.astype(np.float64), rows, 0)[:r]
    return decode_e4m3(q).astype(np.float64) * np.repeat(s, 128, 1)[:, :k]


def block(name: str, a, a_scale, b, b_scale):
    """H, gate and up in float64."""
    x = values(a, a_scale, 1)
    gate, up = (x @ values(b[i], b_scale[i], 128).T for i in (0, 1))
    return act(name, gate) * up, gate, up


def encode_e4m3(y: np.ndarray) -> np.ndarray:
    """Codes of float32 y, to nearest, ties to the even code, saturating."""
    a = np.minimum(np.abs(y).astype(np.float64), 448.0)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1e-30))).astype(np.int64), -6)
    code = ((e + 6) * 8 + np.round(a / 2.0 ** (e - 3))).astype(np.int64)
    return (np.minimum(code, 126) | (np.signbit(y).astype(np.int64) << 7)).astype(np.uint8)


def tiles_1x128(x: np.ndarray):
    """Codes [rows][cols] and scales [cols/128][rows] of float32 values, by the library's contract."""
    t = x.reshape(x.shape[0], -1, 128)
    s = (np.abs(t).max(axis=2) / np.float32(448.0)).astype(np.float32)
    y = (t / np.where(s > 0, s, np.float32(1))[:, :, None]).astype(np.float32)
    return encode_e4m3(y).reshape(x.shape), s.T.copy()


def gradients(name: str, dh, gate, up):
    """dG and dU in float64."""
    dh, gate, up = (np.asarray(v, np.float64) for v in (dh, gate, up))
    return dh * up * slope(name, gate), dh * act(name, gate)
