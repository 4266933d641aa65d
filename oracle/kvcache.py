"""Plain, slow CPU oracle of the 4-bit key/value cache and its attention.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the product path.  It
shares no code, tables or helpers with the HIP library.

16-bit tensors are numpy float32 arrays that hold fp16 or bfloat16 values, with
the type named beside them ("f16" or "bf16").  The definitions:

K1. a block is 64 consecutive dims of a head's vector; its absmax A is the largest
    |x| that is a number (NaNs are left out), one of the 16-bit values;
K2. code = sign bit | nearest E2M1 magnitude of fl32(|x| * fl32(6 * fl32(1 / A))),
    ties to the even code, saturating at 6; a NaN (of x or of the product) gives
    magnitude 0, a zero block has factor 0;
K3. x' = fl32(E2M1 value * fl32(A / 6));
K4. a slab (one page of one head, P tokens, D = 64 NB) holds the bytes
      K:  32 NB t + 8 NB g + 8 b + r // 2           dim 64 b + 16 g + r, r < 16
      V:  32 NB P + 128 NB (t // 4) + 8 NB m + 8 b + 2 place + r // 2
                                                    dim 64 b + 4 m + r, r < 4
      A of K: 64 NB P + 2 (NB t + b),  A of V: 66 NB P + 2 (NB t + b)
    with place = 0, 2, 1, 3 for t % 4 = 0, 1, 2, 3 and even r in the low nibble;
K5. attention as in ``attention`` below, all of it in float64.
"""

from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

BLOCK = 64
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def bits16(x: np.ndarray, kind: str) -> np.ndarray:
    """uint16 patterns of float32 values that are exact in the 16-bit type."""
    x = np.asarray(x, np.float32)
    if kind == "f16":
        return x.astype(np.float16).view(np.uint16)
    return (x.view(np.uint32) >> 16).astype(np.uint16)


def from_bits16(b: np.ndarray, kind: str) -> np.ndarray:
    b = np.asarray(b, np.uint16)
    if kind == "f16":
        return b.view(np.float16).astype(np.float32)
    return (b.astype(np.uint32) << 16).view(np.float32)


def round16(x: np.ndarray, kind: str) -> np.ndarray:
    """float32 values rounded to the nearest 16-bit value, ties to even."""
    x = np.asarray(x, np.float32)
    if kind == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    out = from_bits16(r, "bf16")
    return np.where(np.isnan(x), np.float32(np.nan), out)


def quantize(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(codes uint8 [..., D], A float32 [..., D / 64]) per K1-K2."""
    x = np.asarray(x, np.float32)
    w = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    mag = np.abs(w)
    a = np.where(np.isnan(mag), np.float32(0), mag).max(-1)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        inv = np.where(a > 0, np.float32(6) * (np.float32(1) / a), np.float32(0)).astype(np.float32)
        f = (mag * inv[..., None]).astype(np.float32).astype(np.float64)
        f = np.where(np.isnan(f), 0.0, np.minimum(f, 6.0))
    code = np.zeros(f.shape, np.uint8)
    best = np.full(f.shape, np.inf)
    for c, value in enumerate(MAGNITUDES):
        d = np.abs(f - value)
        take = (d < best) | ((d == best) & (c % 2 == 0))
        code[take], best[take] = c, d[take]
    code |= (np.signbit(w).astype(np.uint8) << 3)
    return code.reshape(x.shape), a


def dequantize(codes: np.ndarray, a: np.ndarray) -> np.ndarray:
    """float32 x' per K3."""
    value = np.array(MAGNITUDES + tuple(-m for m in MAGNITUDES), np.float32)[codes]
    with np.errstate(invalid="ignore"):
        step = (np.asarray(a, np.float32) / np.float32(6)).astype(np.float32)
        v = value.reshape(*codes.shape[:-1], codes.shape[-1] // BLOCK, BLOCK) * step[..., None]
    return v.astype(np.float32).reshape(codes.shape)


def slab_bytes(page: int, d: int) -> int:
    return page * 68 * (d // 64)


def _places(t: int, page: int, d: int, values: bool):
    """Byte of every dim, nibble shift of every dim, first byte of every block's A (K4)."""
    nb = d // 64
    dim = np.arange(d)
    b = dim // 64
    if values:
        place = (0, 2, 1, 3)[t % 4]
        r = dim % 4
        byte = 32 * nb * page + 128 * nb * (t // 4) + 8 * nb * (dim % 64 // 4) + 8 * b + 2 * place + r // 2
    else:
        r = dim % 16
        byte = 32 * nb * t + 8 * nb * (dim % 64 // 16) + 8 * b + r // 2
    scale = (66 if values else 64) * nb * page + 2 * (nb * t + np.arange(nb))
    return byte, 4 * (r % 2), scale


def write(data: np.ndarray, page: int, k: np.ndarray, v: np.ndarray, slots, kind: str) -> None:
    """data uint8 [pages, heads, slab] updated in place."""
    pages, heads, _ = data.shape
    d = k.shape[2]
    (ck, ak), (cv, av) = quantize(k), quantize(v)
    for i, slot in enumerate(int(s) for s in slots):
        if not 0 <= slot < pages * page:
            continue
        for values, code, a in ((False, ck, ak), (True, cv, av)):
            byte, shift, scale = _places(slot % page, page, d, values)
            ab = bits16(a[i], kind)
            for h in range(heads):
                s = data[slot // page, h]
                s[byte] = 0
                np.bitwise_or.at(s, byte, (code[i, h].astype(np.int64) << shift).astype(np.uint8))
                s[scale], s[scale + 1] = ab[h] & 255, ab[h] >> 8


def read(data: np.ndarray, page: int, d: int, slots, kind: str) -> Tuple[np.ndarray, np.ndarray]:
    """float32 k', v' [slots, heads, d]; zeros for a slot outside the cache."""
    pages, heads, _ = data.shape
    out = np.zeros((2, len(slots), heads, d), np.float32)
    for i, slot in enumerate(int(s) for s in slots):
        if not 0 <= slot < pages * page:
            continue
        for n, values in enumerate((False, True)):
            byte, shift, scale = _places(slot % page, page, d, values)
            s = data[slot // page]
            code = (s[:, byte].astype(np.int64) >> shift) & 15
            a = from_bits16(s[:, scale].astype(np.uint16) | (s[:, scale + 1].astype(np.uint16) << 8), kind)
            out[n, i] = dequantize(code.astype(np.uint8), a)
    return out[0], out[1]


def visible(p: int, length: int, window: int, prefix: int) -> np.ndarray:
    j = np.arange(length)
    if p < 0:
        return np.zeros(length, bool)
    return (j < prefix) | ((j <= p) & ((window == 0) | (p - j < window)))


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, window: int = 0, softcap: float = 0.0,
              alibi: Optional[np.ndarray] = None, prefix: int = 0, hidden: Optional[np.ndarray] = None):
    """One sequence in float64: q [n, q_heads, d], k and v [length, heads, d] (x'), hidden bool [length].

    Returns out, lse, and for the bounds on rounding errors sum_j p_j |v_j| [n, q_heads, d]
    and the largest scale * sum |q||k| over visible keys [n, q_heads]."""
    n, q_heads, d = q.shape
    length, heads, _ = k.shape
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    out, size = np.zeros((n, q_heads, d)), np.zeros((n, q_heads, d))
    lse, reach = np.full((n, q_heads), -np.inf), np.zeros((n, q_heads))
    for i in range(n):
        p = length - n + i
        see = visible(p, length, window, prefix)
        if hidden is not None:
            see &= ~hidden
        j = np.nonzero(see)[0]
        if j.size == 0:
            continue
        for h in range(q_heads):
            kk, vv = k[j, h // (q_heads // heads)], v[j, h // (q_heads // heads)]
            s = scale * (kk @ q[i, h])
            reach[i, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[i, h]))).max()
            if softcap:
                s = softcap * np.tanh(s / softcap)
            if alibi is not None:
                s = s - float(alibi[h]) * np.abs(p - j)
            top = s.max()
            e = np.exp(s - top)
            lse[i, h] = top + np.log(e.sum())
            out[i, h], size[i, h] = (e / e.sum()) @ vv, (e / e.sum()) @ np.abs(vv)
    return out, lse, size, reach
