"""Pins of the 4-bit cache's oracle: the byte layout rebuilt another way, hand-worked
blocks, rounding at the ties, and attention against closed forms."""

import numpy as np
import pytest

from oracle import kvcache as kv


def test_layout_is_a_bijection_and_tokens_own_their_bytes():
    for page in (16, 64):
        for d in (64, 128, 256):
            owner = np.full(kv.slab_bytes(page, d), -1)
            for t in range(page):
                for values in (False, True):
                    byte, shift, scale = kv._places(t, page, d, values)
                    own = np.concatenate([np.unique(byte), scale, scale + 1])
                    assert own.size == d // 2 + 2 * (d // 64)
                    assert np.all(owner[own] == -1)
                    owner[own] = t
                    assert len({(int(a), int(b)) for a, b in zip(byte, shift)}) == d
            assert np.all(owner >= 0)


def test_layout_as_nested_arrays():
    page, d = 32, 128
    rng = np.random.default_rng(1)
    k, v = (kv.round16(rng.standard_normal((page, 1, d)), "f16") for _ in range(2))
    data = np.zeros((1, 1, kv.slab_bytes(page, d)), np.uint8)
    kv.write(data, page, k, v, range(page), "f16")
    half = page * d // 2
    (ck, ak), (cv, av) = kv.quantize(k), kv.quantize(v)

    def nibbles(b):
        return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)

    got = nibbles(data[0, 0, :half].reshape(page, 4, 2, 8)).transpose(0, 2, 1, 3).reshape(page, d)
    assert np.array_equal(got, ck[:, 0])
    raw = nibbles(data[0, 0, half:2 * half].reshape(page // 4, 16, 2, 4, 2))[:, :, :, [0, 2, 1, 3]]
    assert np.array_equal(raw.transpose(0, 3, 2, 1, 4).reshape(page, d), cv[:, 0])
    a = data[0, 0, 2 * half:].view(np.float16).reshape(2, page, 2)
    assert np.array_equal(a[0], ak[:, 0].astype(np.float16)) and np.array_equal(a[1], av[:, 0].astype(np.float16))
    rk, rv = kv.read(data, page, d, range(page), "f16")
    assert np.array_equal(rk, kv.dequantize(ck, ak)) and np.array_equal(rv, kv.dequantize(cv, av))


def test_hand_worked_block():
    x = np.zeros(64, np.float32)
    x[:12] = [6, -6, 3, -3, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, np.float32(-0.0)]
    codes, a = kv.quantize(x)
    assert a.tolist() == [6.0]                        # factor fl32(6 * fl32(1 / 6)) = 1
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    assert codes[:12].tolist() == [7, 15, 5, 13, 0, 2, 2, 4, 4, 6, 6, 8]
    assert kv.dequantize(codes, a)[:12].tolist() == [6, -6, 3, -3, 0, 1, 1, 2, 2, 4, 4, 0]


def test_not_numbers_and_zero_blocks():
    x = np.ones((3, 64), np.float32)
    x[0, 3] = np.nan
    x[1, 5] = np.inf
    x[2] = 0
    codes, a = kv.quantize(x)
    assert a.ravel().tolist() == [1.0, np.inf, 0.0]
    assert codes[0, 3] == 0 and np.all(np.delete(codes[0], 3) == 7)
    assert np.all(codes[1] == 0) and np.all(codes[2] == 0)
    got = kv.dequantize(codes, a)
    assert np.all(np.isnan(got[1])) and np.all(got[2] == 0)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_round_trip_error_is_half_a_gap(kind):
    rng = np.random.default_rng(2)
    x = kv.round16(rng.standard_normal((50, 128)) * np.exp(rng.standard_normal((50, 1)) * 3), kind)
    codes, a = kv.quantize(x)
    got = kv.dequantize(codes, a).reshape(50, 2, 64)
    unit = a[..., None] / 6.0
    v = np.abs(x.reshape(50, 2, 64)) / unit
    gap = np.where(v <= 2, 0.5, np.where(v <= 4, 1.0, 2.0))
    assert np.all(np.abs(got - x.reshape(50, 2, 64)) <= (gap / 2 + 1e-5) * unit)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_bits(kind):
    b = np.arange(0, 1 << 16, 7, dtype=np.uint16)
    x = kv.from_bits16(b, kind)
    keep = ~np.isnan(x)
    assert np.array_equal(kv.bits16(x[keep], kind), b[keep])
    assert np.array_equal(kv.round16(x[keep], kind), x[keep])


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 9, 2, 64))
    q = np.zeros((3, 4, 64))
    out, lse, size, reach = kv.attention(q, k, v, 0.125)
    for i in range(3):                                 # equal scores: the mean of what is seen
        n = 9 - 3 + i + 1
        assert np.allclose(lse[i], np.log(n))
        for h in range(4):
            assert np.allclose(out[i, h], v[:n, h // 2].mean(0))
    out, lse, _, _ = kv.attention(q, k, v, 0.125, window=2)
    assert np.allclose(out[2, 0], v[7:, 0].mean(0)) and np.allclose(lse, np.log(2))
    out, lse, _, _ = kv.attention(q, k, v, 0.125, window=2, prefix=3)
    assert np.allclose(out[2, 3], v[[0, 1, 2, 7, 8], 1].mean(0)) and np.allclose(lse, np.log(5))
    out, lse, _, _ = kv.attention(q, k, v, 0.125, alibi=np.full(4, 1e3))
    assert np.allclose(out[:, 0], v[6:, 0]) and np.allclose(lse, 0)    # only the query's own token counts
    q = rng.standard_normal((1, 2, 64))
    out, lse, _, _ = kv.attention(q, k[:1], v[:1], 0.5)
    assert np.allclose(out[0, 1], v[0, 1]) and np.isclose(lse[0, 1], 0.5 * k[0, 1] @ q[0, 1])
    out, lse, _, _ = kv.attention(1e6 * q, k[:1], v[:1], 0.5, softcap=7.0)
    assert np.allclose(np.abs(lse), 7.0)


def test_attention_of_rows_that_see_nothing():
    q = np.ones((4, 1, 64))
    k = v = np.ones((2, 1, 64))
    out, lse, _, _ = kv.attention(q, k, v, 1.0, prefix=2)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(out[2:] == 1)
    out, lse, _, _ = kv.attention(q[:1], k[:0], v[:0], 1.0)
    assert np.all(out == 0) and np.all(np.isneginf(lse))
