"""Pins of the microscaled matrices' oracle: brute force in exact rationals, closed forms."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import mx4

GRID = [Fraction(v) for v in (0, "1/2", 1, "3/2", 2, 3, 4, 6)]


def brute(block):
    """(codes, byte) of 32 finite floats in exact arithmetic."""
    x = [Fraction(float(v)) for v in block]
    top = max(abs(v) for v in x)
    e = -127
    if top > 0:
        f = -2000
        while Fraction(2) ** (f + 1) <= top:
            f += 1
        e = max(f - 2, -127)
    codes = []
    for v, raw in zip(x, block):
        f = min(abs(v) / Fraction(2) ** e, Fraction(6))
        d = [abs(f - g) for g in GRID]
        best = [i for i in range(8) if d[i] == min(d)]
        pick = [i for i in best if i % 2 == 0] or best
        codes.append(pick[0] + (8 if np.signbit(raw) else 0))
    return codes, e + 127


@pytest.mark.parametrize("kind", ["normal", "wide", "ties", "tiny", "huge"])
def test_quantize_matches_exact_rationals(kind):
    rng = np.random.default_rng([71, len(kind)])
    for i in range(20):
        x = rng.standard_normal(32)
        if kind == "wide":
            x *= np.exp2(rng.integers(-12, 12, 32))
        x = x.astype(np.float16).astype(np.float64)
        if kind == "ties":
            x = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, -0.25, -5.0, -0.0, 4.0], 32) * 2.0 ** i
        if kind == "tiny":
            x *= 2.0 ** -126
        if kind == "huge":
            x *= 2.0 ** 120
        codes, scales = mx4.quantize(x[None])
        want, byte = brute(x)
        assert scales[0, 0] == byte and codes[0, :32].tolist() == want


def test_padding_zeros_and_odd_blocks():
    x = np.zeros((4, 100))
    x[1, 40] = np.nan
    x[2, 99] = -np.inf
    x[3] = -0.0
    codes, scales = mx4.quantize(x)
    assert codes.shape == (4, 128) and scales.shape == (4, 4)
    assert scales.tolist() == [[0, 0, 0, 0], [0, 255, 0, 0], [0, 0, 0, 255], [0, 0, 0, 0]]
    assert (codes[:3] == 0).all() and (codes[3, :100] == 8).all() and (codes[3, 100:] == 0).all()
    v = mx4.values(codes, scales)
    assert np.isnan(v[1, 32:64]).all() and np.isfinite(v[1, :32]).all() and np.isnan(v[2, 96:]).all()


def test_values_of_the_grid_come_back():
    for e in (-126, -3, 0, 5, 120):
        x = np.concatenate([mx4.GRID, -mx4.GRID, mx4.GRID, -mx4.GRID]) * 2.0 ** e
        codes, scales = mx4.quantize(x[None])
        assert scales[0, 0] == e + 127
        assert np.array_equal(mx4.values(codes, scales)[0, :32], x)
    assert np.array_equal(mx4.unpack(mx4.pack(codes)), codes)


def test_rotation_closed_forms():
    rng = np.random.default_rng(72)
    x = rng.standard_normal((3, 2, 64))
    one, zero = np.ones((3, 16)), np.zeros((3, 16))
    for inter in (False, True):
        assert np.array_equal(mx4.rotate(x, one, zero, inter), x)
        quarter = mx4.rotate(x, zero, one, inter)
        back = mx4.rotate(quarter, zero, -one, inter)
        assert np.array_equal(back, x)
        assert np.array_equal(quarter[..., 32:], x[..., 32:])
    assert np.array_equal(mx4.rotate(x, zero, one, False)[..., :16], -x[..., 16:32])
    assert np.array_equal(mx4.rotate(x, zero, one, True)[..., 0:32:2], -x[..., 1:32:2])
