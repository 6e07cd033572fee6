"""CPU model of the optimizer step (numpy): in float32, one IEEE rounding per
operation, which the GPU reproduces bit for bit; and the formula in float64."""
from __future__ import annotations

import numpy as np

BLOCK = 128
F = np.float32
_M32 = np.uint64(0xFFFFFFFF)


def decode_e4m3(codes: np.ndarray) -> np.ndarray:
    """float32 values of E4M3 codes (127 and 255: NaN)."""
    c = codes.astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, f * 2.0 ** -9, (8.0 + f) * 2.0 ** (e - 10.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c >= 128, -mag, mag).astype(F)


def mix(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, np.uint64)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B9)) & _M32
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x6A09E667)) & _M32
    return x ^ (x >> np.uint64(16))


def random_bits(numel: int, place: int, step: int, seed: int, first: int = 0) -> np.ndarray:
    """The 32 random bits of `numel` elements, from number `first` on, of the tensor at `place` of a call. (They lie in
    one range of 2^32 element numbers.)"""
    key = np.uint64(seed & 0xFFFFFFFF)
    for v in (seed >> 32, step & 0xFFFFFFFF, place, first >> 32):
        key = (mix(key) + np.uint64(v)) & _M32
    at = (np.arange(numel, dtype=np.uint64) + np.uint64(first)) & _M32
    return mix(at ^ mix(key))


def stochastic_e4m3(y: np.ndarray, bits16: np.ndarray) -> np.ndarray:
    """Magnitude codes of 0 <= y <= 448, up with the probability of what is cut off (in 2^-16 parts)."""
    y = np.minimum(y.astype(np.float64), 448.0)
    e = np.maximum(np.floor(np.log2(np.where(y > 0, y, 1e-30))).astype(np.int64), -6)
    unit = y / 2.0 ** (e - 3)                     # exact: 0 <= unit < 16, the code's last place is 1
    below = np.floor(unit)
    up = np.floor((unit - below) * 2.0 ** 20) + bits16.astype(np.float64) * 16 >= 2.0 ** 20
    value = (below + up).astype(np.int64)         # 8..16 for normal codes, 0..8 below 2^-6
    return np.minimum((e + 6) * 8 + value, 126).astype(np.uint8)


def encode(x: np.ndarray, bits16: np.ndarray, root: bool):
    """Codes and block scales of one tensor's new state."""
    pad = -len(x) % BLOCK
    b = np.pad(np.abs(x), (0, pad)).reshape(-1, BLOCK)
    top = b.max(axis=1)  # (the scale is a product, by the header: it may differ from top / 448 in the last place)
    scale = np.where(np.isfinite(top), top * F(1.0 / 448.0), F(np.nan)).astype(F)
    y = (b / np.where(scale > 0, scale, F(1)).astype(F)[:, None]).reshape(-1)[:len(x)]
    code = stochastic_e4m3(y, bits16)
    if root:
        code = np.where((code == 0) & (x > 0), 1, code).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7), scale


def factors(lr, weight_decay, beta1, beta2, step):
    return (F(1.0 - lr * weight_decay), F(lr / (1.0 - beta1 ** step)), F(1.0 / np.sqrt(1.0 - beta2 ** step)))


def bf16(x: np.ndarray) -> np.ndarray:
    """The bits of x rounded to bf16, ties to even (finite x)."""
    u = x.astype(F).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def step32(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step, grad_scale=1.0):
    """New p, m, root and v of float32 arrays, one rounding per operation."""
    decay, size, root_by = factors(lr, weight_decay, beta1, beta2, step)
    g = g * F(grad_scale)
    m = m * F(beta1) + g * F(1.0 - beta1)
    v = v * F(beta2) + (g * g) * F(1.0 - beta2)
    r = np.sqrt(v)
    return p * decay - (m / (r * root_by + F(eps))) * size, m, r, v


def step64(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step, grad_scale=1.0):
    """New p, m and v by the formula, in float64."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    g = g * grad_scale
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    up = (m / (1.0 - beta1 ** step)) / (np.sqrt(v / (1.0 - beta2 ** step)) + eps)
    return p - lr * weight_decay * p - lr * up, m, v
