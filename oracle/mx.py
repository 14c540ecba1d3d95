"""Microscaled (MX) 4-bit matrices and rotary appending, in 64 bits, from their definitions.

Blocks of 32 consecutive entries of a row share the scale 2^e, e = floor(log2 m) - 2 with m the largest finite
magnitude, between -127 and 127 (-127 for zeros).  Entry x is kept as the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 to
|x| 2^-e (ties to the even place in that list, 6 beyond 6), with its sign; NaN as 0.  A record of 8704 bytes holds 128
rows x 128 entries: scale bytes e + 127, then codes.
"""

from __future__ import annotations

import numpy as np

BLOCK, PIECE, RECORD = 32, 128, 8704
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _blocks(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    n, w = x.shape
    b = np.zeros((n, -(-w // BLOCK) * BLOCK))
    b[:, :w] = x
    return b.reshape(n, -1, BLOCK)


def quantise(x: np.ndarray):
    """Rows x [n][w] -> (codes [n][blocks][32] 0..15, scale bytes [n][blocks])."""
    b = _blocks(x)
    finite = np.isfinite(b)
    top = np.where(finite, np.abs(b), 0).max(-1)
    e = np.where(top > 0, np.frexp(top)[1] - 3, -127).clip(-127, 127)
    with np.errstate(invalid="ignore"):
        a = np.ldexp(np.where(np.isnan(b), 0.0, np.abs(b)), -e[..., None])
    dist = np.abs(np.minimum(a, 6.0)[..., None] - LEVELS)
    near = dist == dist.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    place = np.where(near.sum(-1) == 1, near.argmax(-1), even.argmax(-1))
    sign = np.signbit(b) & ~np.isnan(b)
    return (place + 8 * sign).astype(np.uint8), (e + 127).astype(np.uint8)


def kept(x: np.ndarray) -> np.ndarray:
    """What the 4-bit form keeps of rows x."""
    code, byte = quantise(x)
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0) * 2.0 ** (byte[..., None].astype(np.float64) - 127)
    return v.reshape(len(v), -1)[:, : np.shape(x)[1]]


def scale_at(r, b):
    return (r % 32) * 16 + (r // 32) * 4 + b


def code_at(r, b):
    return 512 + (r // 8) * 512 + b * 128 + (r % 8) * 16


def write(data: np.ndarray, x: np.ndarray) -> None:
    """Writes rows x in their 4-bit form into the bytes ``data``; what lies beyond the rows stays as it is."""
    code, byte = quantise(x)
    n, blocks = byte.shape
    pieces = -(-blocks // 4)
    for r in range(n):
        for b in range(4 * pieces):
            base = ((r // PIECE) * pieces + b // 4) * RECORD
            c = code[r, b] if b < blocks else np.zeros(BLOCK, np.uint8)
            at = base + code_at(r % PIECE, b % 4)
            data[at:at + 16] = c[0::2] | c[1::2] << 4
            data[base + scale_at(r % PIECE, b % 4)] = byte[r, b] if b < blocks else 0


def rotated(x: np.ndarray, positions: np.ndarray, axis: np.ndarray, theta: float) -> np.ndarray:
    """Rows x [n][heads][hd] turned by positions [axes][n]."""
    half = x.shape[-1] // 2
    # the remainder of turns with the integer part of position * frequency taken off exactly enough: long double
    freq = np.power(np.longdouble(theta), -2 * np.arange(half, dtype=np.longdouble) / (2 * half))
    ang = positions[axis].T.astype(np.longdouble) * freq
    c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    a, b = x[..., :half].astype(np.float64), x[..., half:].astype(np.float64)
    return np.concatenate([a * c - b * s, b * c + a * s], -1)
