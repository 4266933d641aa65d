"""The 4-bit cache and its attention at the edges of their ranges, against the CPU
oracle: caps of any size, rows that see no number, values of very different sizes,
blocks of the smallest bfloat16 numbers.

Bounds are those of test_gpu_kvcache.py with e, the error of a score, free of the cap:
the tanh is within 2^-19 of its value (a polynomial of five terms, or 1 - 2 / (1 + e^2y)
at |y| > 1/2 where its roundings, 2^-21, are at most 2^-20 of it), which is 32 of the
2^-24 of scale * sum |q||k'| that 260 of the products' roundings are counted in.
"""

import numpy as np
import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from gpu_util import host, say
from oracle import kvcache as kv
from test_gpu_kvcache import build, dev, dev16, draw, make_cache, wide

pytestmark = pytest.mark.gpu


def check(out, lse, seqs, scale, kind, window=0, softcap=0.0, alibi=None, prefix=None, heads=None):
    """out, lse against the oracle over seqs = [(q, k', v')] (of the named kv heads' rows)."""
    u, least = (2.0 ** -11, 2.0 ** -23) if kind == "f16" else (2.0 ** -8, 0.0)
    got, got_l = wide(out).astype(np.float64), host(lse).astype(np.float64)
    row = 0
    for n, (q, k, v) in enumerate(seqs):
        o, l, size, reach = kv.attention(q, k, v, scale, window, softcap, alibi, 0 if prefix is None else int(prefix[n]))
        far = 0.0 if alibi is None else float(np.abs(alibi).max()) * max(len(k), 1)
        e = 2.0 ** -24 * (260 + 32) * reach + 2.0 ** -20 + 2.0 ** -22 * far
        g, gl = got[row:row + len(q)], got_l[row:row + len(q)]
        row += len(q)
        nothing = np.isneginf(l)
        assert np.array_equal(np.isneginf(gl), nothing), (n, "which rows see nothing")
        el = np.abs(gl[~nothing] - l[~nothing]) - (e[~nothing] + 2.0 ** -21 * np.abs(l[~nothing]))
        assert el.size == 0 or el.max() <= 0, f"sequence {n}: lse off by {el.max()} more than its bound"
        tol = u * np.abs(o) + (u + 2 * e[..., None]) * size + least
        bad = ~(np.abs(g - o) <= tol)
        assert not bad.any(), (f"sequence {n}: {int(bad.sum())} of {bad.size} outside; first at {tuple(np.argwhere(bad)[0])}: "
                               f"{g[bad][0]} oracle {o[bad][0]} bound {tol[bad][0]}")
    assert row == got.shape[0]


@pytest.mark.parametrize("cap", [1e-45, 1e-3, 0.7, 7.0, 50.0, 1e3, 1e5, 1e8, 3e38])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_caps_of_any_size(cap, kind):
    """A cap far above the scores leaves them as they are, one far below makes them equal."""
    for lens, group, d in (([(1, 300), (1, 77)], 4, 128), ([(40, 90)], 1, 64), ([(3, 50)], 2, 256)):
        c, table, lengths, seqs = build(lens, 2, group, d, 32, kind, 40)
        counts = [n for n, _ in lens]
        q = dev16(np.concatenate([s[0] for s in seqs]), kind)
        say(f"fp4_cache_attention capped at {cap}, {lens} {kind}")
        out, lse = i8.fp4_cache_attention(q, c, table, lengths, dev(np.concatenate([[0], np.cumsum(counts)]), torch.int32),
                                          max(counts), scale=0.5, softcap=cap, return_lse=True)
        torch.cuda.synchronize()
        check(out, lse, seqs, 0.5, kind, softcap=float(np.float32(cap)))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("n", [40, 700, 5000], ids=["one_tile", "whole", "cut"])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_log_sum_exp_of_rows_that_meet_no_number(n, kind, softcap):
    """A key that holds an infinity, or a query that does: out and lse are NaN where it is in sight, and only there."""
    rng = np.random.default_rng(41)
    heads, group, d, page = 2, 2, 64, 32
    q, k, v = draw(rng, (3, heads * group, d), kind), draw(rng, (n, heads, d), kind, 0.3), draw(rng, (n, heads, d), kind)
    k[n - 2, 1, 7] = np.inf                    # seen by the last two queries, heads 2 and 3
    q[0, 0, 5] = np.nan
    c = make_cache(-(-n // page) + 1, heads, d, page, kind)
    table = dev(np.arange(-(-n // page))[None], torch.int32)
    say(f"fp4_cache_attention with scores that are no numbers, {n} keys {kind} cap {softcap}")
    i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), torch.arange(n, device="cuda"))
    lengths = dev(np.array([n]), torch.int32)
    out, lse = i8.fp4_cache_attention(dev16(q, kind), c, table, lengths, max_q=3, softcap=softcap, return_lse=True)
    one, one_lse = i8.fp4_cache_attention(dev16(q[:1], kind), c, table, lengths, max_q=1, softcap=softcap, window=2,
                                          return_lse=True)
    none, none_lse = i8.fp4_cache_attention(dev16(q, kind), c, table, 0 * lengths, max_q=3, return_lse=True)
    torch.cuda.synchronize()
    want = np.zeros((3, 4), bool)
    want[0, 0] = want[1:, 2:] = True
    assert np.array_equal(np.isnan(host(lse)), want) and np.isfinite(host(lse)[~want]).all()
    assert np.array_equal(np.isnan(wide(out)).all(-1), want) and np.array_equal(np.isnan(wide(out)).any(-1), want)
    assert np.array_equal(np.isnan(host(one_lse))[0], [True, False, True, True])
    assert np.array_equal(np.isnan(wide(one)).all(-1)[0], [True, False, True, True])
    assert bool((none == 0).all()) and bool(torch.isneginf(none_lse).all())


SPREADS = {
    # log2 of the sizes of V's blocks by key and block, and where the scores lean to
    "block": lambda j, b: np.where(b == 0, 12.0, -10.0) + 0 * j,
    "first_key": lambda j, b: np.where(j == 0, 14.0, -9.0) + 0 * b,
    "last_key": lambda j, b: np.where(j == j.max(), 14.0, -9.0) + 0 * b,
    "small_key": lambda j, b: np.where(j == 5, -10.0, 13.0) + 0 * b,
    "small_last": lambda j, b: np.where(j == j.max(), -10.0, 13.0) + 0 * b,
    "every_other": lambda j, b: np.where(j % 2 == 0, 14.0, -10.0) + 0 * b,
    "falling": lambda j, b: 15.0 - 27.0 * j / j.max() + 0 * b,
    "rising": lambda j, b: 27.0 * j / j.max() - 12.0 + 0 * b,
}


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("lean", [24.0, 7.0], ids=["none", "some"])
@pytest.mark.parametrize("spread", SPREADS)
def test_values_of_very_different_sizes(spread, lean, kind):
    """The keys that draw a row's weight hold values 2^20 and more below others' that draw none, or about e^-20 of it."""
    rng = np.random.default_rng([42, len(spread)])
    heads, d, page = 1, 128, 32
    for n, queries in ((100, 1), (700, 1), (700, 20), (700, 45), (5000, 1)):
        j, b = np.arange(n)[:, None], np.arange(2)[None]
        size = np.asarray(SPREADS[spread](j, b), np.float64)
        q = draw(rng, (queries, heads, d), kind, 0.1)
        along = q[0, 0] / np.abs(q[0, 0]).max()
        to = np.where(size.min(1) < 0, lean, -lean)       # keys of small values draw the weight
        k = kv.round16(to[:, None, None] * along * 0.3 + 0.1 * rng.standard_normal((n, heads, d)), kind)
        q[:] = q[0]
        v = kv.round16(np.clip(rng.standard_normal((n, heads, 2, 64)) * 0.4, -1, 1) * np.exp2(size)[:, None, :, None], kind)
        v = v.reshape(n, heads, d)
        c = make_cache(-(-n // page), heads, d, page, kind)
        say(f"fp4_cache_attention, {spread} values, lean {lean}, {n} keys, {queries} queries {kind}")
        i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), torch.arange(n, device="cuda"))
        out, lse = i8.fp4_cache_attention(dev16(q, kind), c, dev(np.arange(-(-n // page))[None], torch.int32),
                                          dev(np.array([n]), torch.int32), max_q=queries, return_lse=True)
        torch.cuda.synchronize()
        check(out, lse, [(q, kv.dequantize(*kv.quantize(k)), kv.dequantize(*kv.quantize(v)))], d ** -0.5, kind)


@pytest.mark.parametrize("mask", [dict(window=20), dict(window=20, softcap=30.0), dict()], ids=["window", "cap", "causal"])
def test_hidden_keys_of_large_values(mask):
    """Keys out of sight, in the tiles of those in sight, hold values 2^24 above them."""
    rng = np.random.default_rng(43)
    heads, d, page, n, kind = 2, 64, 64, 90, "f16"
    for queries in (1, 18, 50):
        q = draw(rng, (queries, heads, d), kind, 0.3)
        k, v = draw(rng, (n, heads, d), kind, 0.3), draw(rng, (n, heads, d), kind, 0.3) * 2.0 ** -8
        seen = n - 1 if mask else n - queries           # the first query's last key
        big = np.arange(seen - 22, seen - 20) if mask else np.arange(seen + 1, n)
        v[big] = kv.round16(np.clip(v[big] * 2.0 ** 24, -6e4, 6e4), kind)
        v = kv.round16(v, kind)
        c = make_cache(2, heads, d, page, kind)
        say(f"fp4_cache_attention with large values out of sight, {queries} queries {mask}")
        i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), torch.arange(n, device="cuda"))
        out, lse = i8.fp4_cache_attention(dev16(q, kind), c, dev(np.array([[0, 1]]), torch.int32),
                                          dev(np.array([n]), torch.int32), max_q=queries, return_lse=True, **mask)
        torch.cuda.synchronize()
        check(out, lse, [(q, kv.dequantize(*kv.quantize(k)), kv.dequantize(*kv.quantize(v)))], d ** -0.5, kind, **mask)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_write_blocks_of_the_smallest_numbers(d):
    """bfloat16 blocks whose factor 6 / A passes the largest fp32 number: every byte is the oracle's."""
    rng = np.random.default_rng([44, d])
    n, page, kind = 64, 16, "bf16"
    top = rng.integers(1, 0x100, (n, 1, 1))             # A: subnormals, and the first normal numbers (0x0080 = 2^-126)
    top[:8, 0, 0] = [1, 2, 0x7F, 0x80, 0xBF, 0xC0, 0xC1, 0xFF]          # 6 / FLT_MAX = 1.76e-38 lies at 0x00c0
    bits = rng.integers(0, 0x10000, (2, n, 1, d)) % (top + 1)
    bits[..., ::64] = top
    bits[..., 3::64] = 0
    bits = bits | np.where(rng.integers(0, 2, bits.shape) > 0, 0x8000, 0)
    k, v = (kv.from_bits16(x.astype(np.uint16), kind) for x in bits)
    say(f"fp4_cache_write of the smallest bfloat16 numbers, head_dim {d}")
    c = make_cache(n // page, 1, d, page, kind)
    want = host(c.data).copy()
    kv.write(want, page, k, v, range(n), kind)
    t = [torch.from_numpy(x.astype(np.uint16).view(np.int16)).view(torch.bfloat16).cuda() for x in bits]
    i8.fp4_cache_write(c, *t, torch.arange(n, device="cuda"))
    got = i8.fp4_cache_read(c, torch.arange(n, device="cuda"), torch.float32)
    torch.cuda.synchronize()
    assert np.array_equal(host(c.data), want)
    for g, r in zip(got, kv.read(want, page, d, range(n), kind)):
        assert np.array_equal(wide(g).view(np.int32), np.asarray(r, np.float32).view(np.int32))


def test_views_that_would_be_read_or_written_past_their_end():
    c = make_cache(4, 1, 64, 16, "f16")
    q = torch.zeros((2, 1, 64), dtype=torch.float16, device="cuda")
    table, lengths = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        i8.fp4_cache_attention(q, c, table[:1].expand(2, 4), lengths)
    for bad in (torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 20), torch.zeros(1 << 20, device="cuda"),
                torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            i8.fp4_cache_attention(q, c, table, lengths, workspace=bad)


def test_values_past_32_bits_are_refused():
    c = make_cache(4, 1, 64, 16, "f16")
    q = torch.zeros((2, 1, 64), dtype=torch.float16, device="cuda")
    table, lengths = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    offsets = torch.arange(3, dtype=torch.int32, device="cuda")
    for bad in (dict(window=(1 << 32) + 1), dict(max_len=(1 << 32) + 16), dict(q_offsets=offsets, max_q=(1 << 32) + 1),
                dict(softcap=1e-50)):
        with pytest.raises(ValueError):
            i8.fp4_cache_attention(q, c, table, lengths, **bad)


@pytest.mark.parametrize("heads,group,d", [(2, 3, 64), (1, 8, 128), (3, 1, 256)])
def test_rows_of_no_sequence(heads, group, d):
    """Padding around the sequences' queries and queries past max_q: zeros and -inf, or what a given out holds."""
    kind, page = "f16", 16
    lens = [(3, 50), (0, 20), (9, 4000), (1, 1), (2, 0)]
    c, table, lengths, seqs = build(lens, heads, group, d, page, kind, 45)
    rows = np.concatenate([s[0] for s in seqs])
    n, hq = len(rows) + 31, heads * group
    q = np.concatenate([np.full((7, hq, d), np.nan), rows, np.full((24, hq, d), np.nan)])
    offsets = dev(7 + np.concatenate([[0], np.cumsum([x for x, _ in lens])]), torch.int32)
    say(f"fp4_cache_attention with rows of no sequence, {heads} x {group} heads of {d}")
    dirty = [torch.full((n * hq * d,), 3.0, dtype=torch.float16, device="cuda") for _ in range(4)]
    dirty += [torch.full((n * hq,), 3.0, device="cuda") for _ in range(4)]
    del dirty                                   # what the call allocates is not zero
    mark = torch.full((n, hq, d), 5.0, dtype=torch.float16, device="cuda")
    for most, out in ((9, None), (2, None), (9, mark.clone()), (2, mark.clone())):
        got, lse = i8.fp4_cache_attention(dev16(q, kind), c, table, lengths, offsets, most, out=out, return_lse=True)
        torch.cuda.synchronize()
        own = np.zeros(n, bool)
        at = 7
        for (count, length), (qs, k, v) in zip(lens, seqs):
            for i in range(min(count, most)):
                own[at + i] = True
                end = length - count + i + 1
                check(got[at + i:at + i + 1], lse[at + i:at + i + 1], [(qs[i:i + 1], k[:max(end, 0)], v[:max(end, 0)])],
                      d ** -0.5, kind)
            at += count
        rest = torch.from_numpy(~own).cuda()
        assert bool((got[rest] == (0.0 if out is None else 5.0)).all()) and bool(torch.isneginf(lse[rest]).all())
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    got, lse = i8.fp4_cache_attention(dev16(q, kind), c, table[:0], none, torch.zeros(1, dtype=torch.int32, device="cuda"), 1,
                                      return_lse=True)
    assert bool((got == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("where", ["one_block", "first_tile", "some_keys", "all"])
def test_blocks_of_zeros(where, kind):
    """Values that are zero (a padded head, padding tokens), alone and among values of ordinary and of very different sizes."""
    rng = np.random.default_rng(47)
    heads, d, page, n = 2, 128, 16, 300
    for queries, spread in ((1, 0), (40, 0), (40, 24)):
        q, k = draw(rng, (queries, heads, d), kind, 0.3), draw(rng, (n, heads, d), kind, 0.3)
        v = draw(rng, (n, heads, d), kind, 0.3)
        if spread:
            v = kv.round16(np.clip(v, -3, 3) * np.exp2(rng.choice([-spread / 2, spread / 2], (n, 1, 1))), kind)
        v[{"one_block": np.s_[:, :, 64:], "first_tile": np.s_[:32], "some_keys": np.s_[::3], "all": np.s_[:]}[where]] = 0
        c = make_cache(-(-n // page), heads, d, page, kind)
        say(f"fp4_cache_attention with zeros in V, {where}, {queries} queries, spread {spread} {kind}")
        i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), torch.arange(n, device="cuda"))
        out, lse = i8.fp4_cache_attention(dev16(q, kind), c, dev(np.arange(-(-n // page))[None], torch.int32),
                                          dev(np.array([n]), torch.int32), max_q=queries, return_lse=True)
        torch.cuda.synchronize()
        check(out, lse, [(q, kv.dequantize(*kv.quantize(k)), kv.dequantize(*kv.quantize(v)))], d ** -0.5, kind)
