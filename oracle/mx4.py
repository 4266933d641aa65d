"""Plain, slow CPU oracle of the microscaled 4-bit matrices and of the rotation by position.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the product path.  It shares no
code, tables or helpers with the HIP library.

The definitions (the OCP microscaling format MXFP4, its conversion from wider types):

X1. elements are E2M1 (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), blocks are 32
    neighbours along k, each under a power of two 2^E held as the byte E + 127;
X2. E = max(floor(log2 max|x|) - 2, -127); a block of zeros has E = -127; a block with
    a NaN or an infinity has the byte 255, codes of 0, and stands for NaNs;
X3. code = sign of x (that of -0 too) | magnitude nearest to |x| / 2^E, ties to the
    even code, at most 6;
X4. rows are padded with zeros to whole multiples of 128 elements; a block of padding
    is a block of zeros;
X5. products are of the values x', in float64 here;
R1. pair i of a head turns by its token's angle: (a cos - b sin, b cos + a sin),
    float64 rounded to fp32 and then to the 16-bit type.
"""

from __future__ import annotations

from typing import Tuple

import numpy as np

BLOCK = 32
PAD = 128
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(codes uint8 [rows, kp], one each, and scale bytes uint8 [rows, kp / 32]) of x [rows, k] (X1-X4)."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    kp = -(-k // PAD) * PAD
    w = np.zeros((rows, kp))
    w[:, :k] = x
    w = w.reshape(rows, kp // BLOCK, BLOCK)
    odd = ~np.isfinite(w).all(-1)
    safe = np.where(odd[..., None], 0.0, w)
    top = np.abs(safe).max(-1, initial=0.0)
    e = np.full(top.shape, -127)
    live = top > 0
    e[live] = np.maximum(np.floor(np.log2(top[live])).astype(int) - 2, -127)
    f = np.abs(safe) / np.exp2(e.astype(np.float64))[..., None]
    f = np.minimum(f, 6.0)
    near = np.abs(f[..., None] - GRID)
    cand = near == near.min(-1, keepdims=True)
    even = cand & (np.arange(8) % 2 == 0)
    code = np.argmax(np.where(even.any(-1, keepdims=True), even, cand), -1)
    code = np.where(odd[..., None], 0, code + 8 * np.signbit(safe))
    return code.astype(np.uint8).reshape(rows, kp), np.where(odd, 255, e + 127).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """x' float64 [rows, kp] of one-byte codes."""
    c = codes.astype(int)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v.reshape(*scales.shape, BLOCK) * s[..., None]).reshape(codes.shape)


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def unpack(data: np.ndarray) -> np.ndarray:
    return np.stack((data & 15, data >> 4), -1).reshape(data.shape[0], -1)


def rounded(x: np.ndarray) -> np.ndarray:
    """x' float64 of x [rows, k]."""
    return values(*quantize(x))[:, :x.shape[1]]


def matmul(a: np.ndarray, b: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(a . b^T, sum of magnitudes) of values a [m, k] and b [n, k]."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """float64 x [tokens, heads, D] whose first 2 * cos.shape[1] dims are turned (R1, not yet rounded)."""
    out = np.array(x, np.float64)
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[:, i, None].astype(np.float64), sin[:, i, None].astype(np.float64)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out
