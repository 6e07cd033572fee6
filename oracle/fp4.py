"""CPU oracle for FP4 microscaling (OCP MX with E2M1 elements): codes, scale
bytes, the tile layout and the product, in float64. TEST INFRASTRUCTURE ONLY,
as the rest of ``oracle``."""
from __future__ import annotations

import numpy as np

# the value of every E2M1 code: sign, two exponent bits (bias 1), one mantissa bit
VALUES = np.array([s * v for s in (1.0, -1.0) for v in (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)])


def bf16_to_f64(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def encode(v: np.ndarray) -> np.ndarray:
    """E2M1 code of each finite float64: the nearest magnitude by search, the
    even code of two equally near ones, 6 past the end."""
    mags = VALUES[:8]
    d = np.abs(np.abs(v)[..., None] - mags)
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def quantize(bits: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """bf16 bits [rows][cols] -> codes uint8 [rows][K] (one per element, K =
    cols rounded up to 32 with zero codes) and E8M0 bytes [rows][K/32]. A block
    with an infinity or NaN: byte 255, zero codes."""
    x = bf16_to_f64(bits)
    rows, cols = x.shape
    k = -(-cols // 32) * 32
    p = np.zeros((rows, k))
    p[:, :cols] = x
    p = p.reshape(rows, k // 32, 32)
    bad = ~np.isfinite(p).all(axis=2)
    p = np.where(bad[..., None], 0.0, p)
    amax = np.abs(p).max(axis=2)
    _, ex = np.frexp(amax)  # amax = m * 2^ex, 0.5 <= m < 1
    e = np.where(amax == 0, -127, np.clip(ex - 1 - 2, -127, 127))
    codes = encode(np.ldexp(p, -e[..., None]))
    codes[bad] = 0
    return codes.reshape(rows, k), np.where(bad, 255, e + 127).astype(np.uint8)


def tiles(codes: np.ndarray, ebytes: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """Codes [rows][K] and bytes [rows][K/32] in the tile layout: q uint8
    [kt][rt][1024], scale uint8 [kg][rt][64][4]."""
    rows, k = codes.shape
    kt, rt = -(-k // 128), -(-rows // 16)
    q = np.zeros((kt, rt, 1024), np.uint8)
    s = np.zeros((-(-kt // 4), rt, 64, 4), np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(k), indexing="ij")
    b = c % 128 // 32
    at = 64 * (r % 16) + 16 * (b ^ (r % 16 >> 2 & 3)) + c % 32 // 2
    np.add.at(q, (c // 128, r // 16, at), (codes << (4 * (c % 2))).astype(np.uint8))
    r, blk = np.meshgrid(np.arange(rows), np.arange(k // 32), indexing="ij")
    s[blk // 16, r // 16, 4 * (r % 16) + blk % 4, blk // 4 % 4] = ebytes
    return q, s


def values(codes: np.ndarray, ebytes: np.ndarray) -> np.ndarray:
    """float64 [rows][K]; NaN where the block's byte is 255."""
    e = np.repeat(ebytes.astype(np.int64) - 127, 32, axis=1)
    v = np.ldexp(VALUES[codes], e)
    return np.where(e == 128, np.nan, v)


def gemm(a: np.ndarray, b: np.ndarray) -> np.ndarray:
    """float64 C[m][n] of two value matrices, unrounded."""
    return a @ b.T
