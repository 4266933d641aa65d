"""GPU parity of the 4-bit key/value cache and its attention against the CPU oracle.

Bit-exact: the cache's bytes after a write (all of them, so that nothing beside the
named slots changed) and what is read back.

Attention, element by element, from the roundings it has (u = 2^-11 for fp16, 2^-8
for bfloat16, the unit roundoff of the output and of the weights e^s A):
  |out - oracle| <= u |out| + (u + 2 e) sum_j p_j |v_j| + t,  |lse - oracle| <= e + 2^-21 |lse|
(fp16 rounds e^s and then e^s A, so one u for both is less than their worst case)
with t = 2^-24 sum of the type's smallest steps (fp16 only) and e the error of a
score in fp32: products of up to 256 terms, summed in any order, err by at most
2^-24 * 260 of scale * sum |q||k'|; 2^-20 covers the exponential, 2^-20 cap the tanh,
2^-22 of the largest distance term the bias.
"""

import ctypes

import numpy as np
import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from gpu_util import host, say
from int8_mixed_precision_vectorwise_amd import _lib
from oracle import kvcache as kv

pytestmark = pytest.mark.gpu

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


def dev16(x, kind):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(DTYPE[kind])


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def wide(t):
    return host(t.float())


def draw(rng, shape, kind, spread=1.0):
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[:-1] + (1,)) * spread)
    return kv.round16(x, kind)


def make_cache(pages, heads, d, page, kind, fill=0xA5):
    c = i8.Fp4Cache.create(pages, heads, d, page, DTYPE[kind])
    c.data.fill_(fill)
    return c


# ---- write and read -------------------------------------------------------------

MOVES = [
    # tokens, heads, d, page, pages, kind
    (1, 1, 64, 16, 1, "f16"),
    (1, 40, 128, 64, 2, "f16"),
    (3, 2, 256, 32, 2, "bf16"),
    (17, 3, 128, 16, 5, "bf16"),
    (65, 2, 64, 256, 2, "f16"),
    (200, 5, 128, 128, 3, "f16"),
    (333, 1, 256, 64, 7, "bf16"),
]


@pytest.mark.parametrize("case", MOVES, ids=lambda c: "t%d_h%d_d%d_p%d_x%d_%s" % c)
@pytest.mark.parametrize("order", ["run", "scattered"])
def test_write_and_read_bit_exact(case, order):
    n, heads, d, page, pages, kind = case
    rng = np.random.default_rng([60, n, heads, d])
    k, v = draw(rng, (n, heads, d), kind), draw(rng, (n, heads, d), kind)
    k[0, 0, :64] = 0
    v[n - 1, heads - 1, 1] = -0.0
    slots = rng.permutation(pages * page)[:n] if order == "scattered" else np.arange(n) + (pages * page - n) // 2
    if n > 10:
        slots[3], slots[7], slots[9] = -1, pages * page, 1 << 40       # none of them in the cache
    say(f"fp4_cache_write {case} {order}")
    c = make_cache(pages, heads, d, page, kind)
    want = host(c.data).copy()
    kv.write(want, page, k, v, slots, kind)
    st = dev(slots, torch.int64)
    i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), st)
    torch.cuda.synchronize()
    got = host(c.data)
    assert np.array_equal(got, want), f"{int((got != want).sum())} of {got.size} bytes differ"
    rk, rv = kv.read(want, page, d, slots, kind)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        say(f"fp4_cache_read {case} {order} {dtype}")
        gk, gv = i8.fp4_cache_read(c, st, dtype)
        torch.cuda.synchronize()
        kind_out = {torch.float16: "f16", torch.bfloat16: "bf16"}.get(dtype)
        for g, r in ((gk, rk), (gv, rv)):
            r = r if kind_out is None else kv.round16(r, kind_out)
            assert np.array_equal(wide(g).view(np.int32), np.asarray(r, np.float32).view(np.int32))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_write_ties_and_not_numbers(kind):
    """Every quotient near a tie, NaNs and infinities, subnormals and the largest values."""
    rng = np.random.default_rng(61)
    d, page, n = 128, 16, 16
    k = kv.round16(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])[rng.integers(0, 8, (n, 1, d))] *
                   rng.choice([-1.0, 1.0], (n, 1, d)) * kv.round16(rng.uniform(0.01, 50, (n, 1, 1)), kind), kind)
    v = kv.round16(rng.integers(-48, 49, (n, 1, d)) / 8.0, kind)
    v[0, 0, 3] = np.nan
    v[1, 0, 70] = np.inf
    v[2, 0, 0] = -np.inf
    v[3, 0] = kv.from_bits16(rng.integers(0, 128, d).astype(np.uint16), kind) if kind == "f16" else 0    # subnormals
    v[4, 0, :] = np.nan
    v[5, 0] = kv.from_bits16(np.uint16(0x7BFF if kind == "f16" else 0x7F7F), kind) * rng.choice([-1, 1], d)
    say(f"fp4_cache_write of ties and NaNs {kind}")
    c = make_cache(1, 1, d, page, kind)
    want = host(c.data).copy()
    kv.write(want, page, k, v, range(n), kind)
    i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), torch.arange(n, device="cuda"))
    torch.cuda.synchronize()
    assert np.array_equal(host(c.data), want)
    gk, gv = i8.fp4_cache_read(c, torch.arange(n, device="cuda"), torch.float32)
    rk, rv = kv.read(want, page, d, range(n), kind)
    assert np.array_equal(wide(gk), rk) and np.array_equal(wide(gv), rv, equal_nan=True)


def test_write_from_strided_views():
    """k and v as parts of a fused projection's output, and head-major tensors."""
    rng = np.random.default_rng(62)
    n, heads, d, page = 37, 3, 128, 32
    x = draw(rng, (n, 3 * heads, d), "f16")
    t = dev16(x, "f16")
    slots = dev(rng.permutation(4 * page)[:n], torch.int64)
    say("fp4_cache_write of strided views")
    a, b = make_cache(4, heads, d, page, "f16"), make_cache(4, heads, d, page, "f16")
    i8.fp4_cache_write(a, t[:, heads:2 * heads], t[:, 2 * heads:], slots)
    hm = t.transpose(0, 1).contiguous()            # [heads, tokens, d]
    i8.fp4_cache_write(b, hm[heads:2 * heads].transpose(0, 1), hm[2 * heads:].transpose(0, 1), slots)
    torch.cuda.synchronize()
    want = np.full_like(host(a.data), 0xA5)
    kv.write(want, page, x[:, heads:2 * heads], x[:, 2 * heads:], host(slots), "f16")
    assert np.array_equal(host(a.data), want) and np.array_equal(host(b.data), want)


@pytest.mark.parametrize("start", range(8))
def test_runs_that_start_inside_a_group_of_four(start):
    """Runs of tokens whose slots are consecutive from any place, with gaps and the runs' joints inside spans of 32."""
    rng = np.random.default_rng([66, start])
    heads, d, page, pages, kind = 3, 64, 16, 14, "f16"
    order = rng.permutation(pages)
    at = np.concatenate([np.arange(70) + start, np.arange(29) + 90 + (start * 3) % 7, np.arange(33) + 140])
    slots = order[at // page] * page + at % page
    slots[[1, 31, 32, 69]] = -1
    slots[50] = pages * page + 3
    n = len(slots)
    k, v = draw(rng, (n, heads, d), kind), draw(rng, (n, heads, d), kind)
    say(f"fp4_cache_write of runs from {start}")
    c = make_cache(pages, heads, d, page, kind)
    want = host(c.data).copy()
    kv.write(want, page, k, v, slots, kind)
    st = dev(slots, torch.int64)
    i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), st)
    got = i8.fp4_cache_read(c, st, torch.float32)
    torch.cuda.synchronize()
    assert np.array_equal(host(c.data), want)
    for g, r in zip(got, kv.read(want, page, d, slots, kind)):
        assert np.array_equal(wide(g).view(np.int32), np.asarray(r, np.float32).view(np.int32))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_calls_larger_than_the_last_level_cache(kind):
    """One call that moves more than 256 MiB gives the bytes and values of small calls (which other tests pin)."""
    heads, d, page, n = 40, 256, 128, 6001
    gen = torch.Generator(device="cuda").manual_seed(67)
    k, v = (torch.randn((n, heads, d), generator=gen, device="cuda").to(DTYPE[kind]) for _ in range(2))
    slots = torch.arange(n, device="cuda") + 2
    slots[700] = -1
    say(f"fp4_cache_write and read of {n} tokens of {heads} heads of {d}, {kind}")
    a, b = (make_cache(-(-(n + 2) // page), heads, d, page, kind) for _ in range(2))
    i8.fp4_cache_write(a, k, v, slots)
    for i in range(0, n, 997):
        i8.fp4_cache_write(b, k[i:i + 997], v[i:i + 997], slots[i:i + 997])
    torch.cuda.synchronize()
    assert torch.equal(a.data, b.data)
    for dtype in (torch.float32, DTYPE[kind]):
        whole = i8.fp4_cache_read(a, slots, dtype)
        for i in range(0, n, 997):
            for x, y in zip(whole, i8.fp4_cache_read(a, slots[i:i + 997], dtype)):
                assert torch.equal(x[i:i + 997], y)


def test_calls_of_more_than_one_launch():
    """Heads and tokens of more than 2^22 workgroups.  Rows that overlap keep the buffers small: every token's keys
    are those of the one before it, moved by a head; the read is of empty slots, which are zeros."""
    heads, d, n = 32768, 256, 4300
    assert -(-n // 32) * 9 * (heads * 32 // 256) > 1 << 22
    gen = torch.Generator(device="cuda").manual_seed(68)
    flat = torch.randn((n + heads) * d, generator=gen, device="cuda").half()
    k = flat.as_strided((n, heads, d), (d, d, 1))
    keep = [0, 1, 2, 3, 1000, 3615, 3616, 3700, n - 2, n - 1]
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    slots[keep] = torch.arange(len(keep), device="cuda") + 3
    say(f"fp4_cache_write of {n} tokens of {heads} heads of {d}")
    a, b = (make_cache(1, heads, d, 16, "f16") for _ in range(2))
    i8.fp4_cache_write(a, k, k, slots)
    i8.fp4_cache_write(b, k[keep].contiguous(), k[keep].contiguous(), slots[keep])
    torch.cuda.synchronize()
    assert torch.equal(a.data, b.data)
    out = torch.full(((n + heads - 1) * d + 64,), 7.0, dtype=torch.float16, device="cuda")
    none = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    c = a.struct()
    say("fp4_cache_read of the same size")
    status = _lib.lib().i8mp_fp4_cache_read(ctypes.byref(c), none.data_ptr(), n, 0, out.data_ptr(), d, d, out.data_ptr(), d,
                                            d, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0 and bool((out[:-64] == 0).all()) and bool((out[-64:] == 7.0).all())


def test_attention_of_more_than_one_launch():
    """A bound on the queries that lays out more than 2^23 workgroups for each sequence."""
    lens, heads, group, d = [(5, 50), (3, 33)], 4, 2, 64
    c, table, lengths, seqs = build(lens, heads, group, d, 16, "f16", 26)
    max_q = 1 << 26
    assert -(-max_q * group // 48) * heads > 1 << 23
    say("fp4_cache_attention with a large bound on the queries")
    out, lse = i8.fp4_cache_attention(dev16(np.concatenate([s[0] for s in seqs]), "f16"), c, table, lengths,
                                      dev(np.array([0, 5, 8]), torch.int32), max_q, return_lse=True)
    torch.cuda.synchronize()
    check(out, lse, seqs, d ** -0.5, "f16")


def test_slots_past_32_bit_offsets():
    """A cache of over 4 GiB: the first and the last pages hold what was written there."""
    heads, d, page = 8, 256, 256
    pages = (1 << 32) // (heads * kv.slab_bytes(page, d)) + 40
    rng = np.random.default_rng(63)
    slots = np.array([0, 5, pages * page - 1, (pages - 1) * page, (pages - 20) * page + 77])
    k, v = draw(rng, (5, heads, d), "bf16"), draw(rng, (5, heads, d), "bf16")
    c = i8.Fp4Cache(torch.empty((pages, heads, kv.slab_bytes(page, d)), dtype=torch.uint8, device="cuda"), page, d,
                    torch.bfloat16)
    assert c.data.numel() > 1 << 32
    say(f"fp4 cache of {c.data.numel()} bytes")
    st = dev(slots, torch.int64)
    i8.fp4_cache_write(c, dev16(k, "bf16"), dev16(v, "bf16"), st)
    gk, gv = i8.fp4_cache_read(c, st, torch.float32)
    torch.cuda.synchronize()
    for g, x in ((gk, k), (gv, v)):
        assert np.array_equal(wide(g), kv.dequantize(*kv.quantize(x)))
    # a sequence on the last page: 5 tokens written to its start, read through the table
    last = np.arange(5) + (pages - 1) * page
    i8.fp4_cache_write(c, dev16(k, "bf16"), dev16(v, "bf16"), dev(last, torch.int64))
    q = draw(rng, (1, heads, d), "bf16")
    out, lse = i8.fp4_cache_attention(dev16(q, "bf16"), c, dev(np.array([[pages - 1]]), torch.int32),
                                      dev(np.array([5]), torch.int32), return_lse=True)
    torch.cuda.synchronize()
    check(out, lse, [(q, kv.dequantize(*kv.quantize(k)), kv.dequantize(*kv.quantize(v)))], d ** -0.5, "bf16")


# ---- attention --------------------------------------------------------------------

def check(out, lse, seqs, scale, kind, window=0, softcap=0.0, alibi=None, prefix=None, hidden=None):
    """out, lse against the oracle over seqs = [(q, k', v')], rows in order, to the bounds above."""
    u = 2.0 ** -11 if kind == "f16" else 2.0 ** -8
    got, got_l = wide(out).astype(np.float64), host(lse).astype(np.float64)
    row = 0
    for n, (q, k, v) in enumerate(seqs):
        o, l, size, reach = kv.attention(q, k, v, scale, window, softcap, alibi, 0 if prefix is None else int(prefix[n]),
                                         None if hidden is None else hidden[n])
        far = 0.0 if alibi is None else float(np.abs(alibi).max()) * max(len(k), 1)
        e = (2.0 ** -24 * 260 * reach + 2.0 ** -20 * (1 + softcap) + 2.0 ** -22 * far)
        g, gl = got[row:row + len(q)], got_l[row:row + len(q)]
        row += len(q)
        nothing = np.isneginf(l)
        assert np.array_equal(np.isneginf(gl), nothing), (n, "which rows see nothing")
        assert np.all(g[nothing] == 0)
        el = np.abs(gl[~nothing] - l[~nothing]) - (e[~nothing] + 2.0 ** -21 * np.abs(l[~nothing]))
        assert el.size == 0 or el.max() <= 0, f"sequence {n}: lse off by {el.max()} more than its bound"
        tol = u * np.abs(o) + (u + 2 * e[..., None]) * size + (2.0 ** -23 if kind == "f16" else 0.0)
        bad = ~(np.abs(g - o) <= tol)
        assert not bad.any(), (f"sequence {n}: {int(bad.sum())} of {bad.size} outside; first at {tuple(np.argwhere(bad)[0])}: "
                               f"{g[bad][0]} oracle {o[bad][0]} bound {tol[bad][0]}")
    assert row == got.shape[0]


def build(lens, heads, group, d, page, kind, seed, garbage=True):
    """A cache that holds sequences of lens = [(queries, length)], its table and inputs."""
    rng = np.random.default_rng([64, seed])
    used = [max(-(-length // page), 0) for _, length in lens]
    pages = sum(used) + 2
    ids = rng.permutation(pages)
    cols = max(used + [1]) + 1
    table = np.full((len(lens), cols), -7)          # unused places name no page
    c = make_cache(pages, heads, d, page, kind, 0xFF if garbage else 0)    # scales that are NaN
    seqs, slots, at = [], [], 0
    ks, vs = [], []
    for i, (n, length) in enumerate(lens):
        table[i, :used[i]] = ids[at:at + used[i]]
        at += used[i]
        k, v = draw(rng, (length, heads, d), kind, 0.3), draw(rng, (length, heads, d), kind, 1.0)
        ks.append(k)
        vs.append(v)
        slots.append(table[i, np.arange(length) // page] * page + np.arange(length) % page)
        q = draw(rng, (n, heads * group, d), kind, 0.3)
        seqs.append((q, kv.dequantize(*kv.quantize(k)), kv.dequantize(*kv.quantize(v))))
    k, v, s = np.concatenate(ks), np.concatenate(vs), np.concatenate(slots)
    i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), dev(s, torch.int64))
    return c, dev(table, torch.int32), dev(np.array([n for _, n in lens]), torch.int32), seqs


def attend(lens, heads, group, d, page, kind, seed, window=0, softcap=0.0, alibi=False, prefix=None, scale=None,
           max_len=None, offsets=True):
    c, table, lengths, seqs = build(lens, heads, group, d, page, kind, seed)
    q = dev16(np.concatenate([s[0] for s in seqs]), kind)
    counts = [n for n, _ in lens]
    qo = dev(np.concatenate([[0], np.cumsum(counts)]), torch.int32) if offsets else None
    slopes = np.exp2(-8.0 * np.arange(1, heads * group + 1) / (heads * group)).astype(np.float32) if alibi else None
    pre = None if prefix is None else np.array(prefix)
    say(f"fp4_cache_attention lens={lens[:4]}.. heads={heads}x{group} d={d} page={page} {kind} window={window} cap={softcap} "
        f"alibi={alibi} prefix={prefix}")
    out, lse = i8.fp4_cache_attention(q, c, table, lengths, q_offsets=qo, max_q=max(counts), max_len=max_len, scale=scale,
                                      window=window, softcap=softcap, alibi=None if slopes is None else dev(slopes, torch.float32),
                                      prefix=None if pre is None else dev(pre, torch.int32), return_lse=True)
    torch.cuda.synchronize()
    check(out, lse, seqs, d ** -0.5 if scale is None else scale, kind, window, softcap, slopes, pre)
    return out


DECODE = [
    # lengths, kv heads, group, d, page, kind
    ([1], 1, 1, 64, 16, "f16"),
    ([2, 15, 16, 17, 31, 32, 33], 2, 1, 128, 16, "f16"),
    ([1, 63, 64, 65, 127, 129], 1, 8, 128, 64, "bf16"),
    ([0, 1, 0, 5], 2, 2, 64, 32, "bf16"),
    ([100, 0, 257], 2, 3, 256, 128, "f16"),
    ([700], 1, 16, 128, 256, "bf16"),
    ([300, 41], 2, 17, 64, 32, "f16"),
    ([70], 1, 40, 128, 16, "bf16"),
    ([1000, 3], 1, 7, 256, 32, "bf16"),
    ([2500], 2, 1, 64, 16, "f16"),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "%s_h%dx%d_d%d_p%d_%s" % ("-".join(map(str, c[0])), *c[1:]))
def test_decode(case):
    lengths, heads, group, d, page, kind = case
    attend([(1, n) for n in lengths], heads, group, d, page, kind, sum(lengths), offsets=False)


QUERIES = [
    # (queries, length) of each sequence, kv heads, group, d, page, kind
    ([(2, 2), (3, 70), (1, 9)], 2, 2, 128, 16, "f16"),
    ([(5, 3), (4, 0), (1, 1)], 1, 4, 64, 32, "bf16"),              # queries before the first token
    ([(8, 40)], 1, 2, 256, 64, "f16"),
    ([(33, 33), (1, 200), (17, 130)], 2, 1, 128, 64, "bf16"),
    ([(100, 100)], 1, 5, 64, 16, "f16"),
    ([(129, 300), (64, 64)], 1, 1, 128, 32, "f16"),
    ([(70, 70), (130, 131)], 1, 2, 256, 16, "bf16"),
    ([(257, 257)], 2, 1, 128, 128, "bf16"),
]


@pytest.mark.parametrize("case", QUERIES, ids=lambda c: "%s_h%dx%d_d%d_p%d_%s" % ("-".join("%dof%d" % p for p in c[0]), *c[1:]))
def test_several_queries(case):
    lens, heads, group, d, page, kind = case
    attend(lens, heads, group, d, page, kind, sum(n for _, n in lens))


@pytest.mark.parametrize("lens", [[(1, 200), (1, 40), (1, 7)], [(6, 150), (3, 3), (2, 90)], [(80, 190), (33, 40)]],
                         ids=["decode", "draft", "prompt"])
@pytest.mark.parametrize("mask", [
    dict(window=1), dict(window=16), dict(window=33, prefix=True), dict(window=50, alibi=True), dict(prefix=True),
    dict(softcap=3.0), dict(softcap=30.0, alibi=True, prefix=True, window=20), dict(scale=0.0), dict(scale=-0.4),
    dict(window=1 << 30)], ids=lambda m: "_".join(m))
def test_masks_and_scores(lens, mask):
    mask = dict(mask)
    if mask.pop("prefix", False):
        mask["prefix"] = [35, 1000, 0][:len(lens)]          # the second reaches past its sequence's end
    for heads, group, d, page, kind in ((1, 4, 128, 16, "f16"), (2, 1, 64, 64, "bf16")):
        attend(lens, heads, group, d, page, kind, 7 + len(mask), **mask)


@pytest.mark.parametrize("lens", [[(1, 20011)], [(1, 9000), (1, 100), (1, 0), (1, 4097)], [(4, 6001), (2, 500)]])
def test_keys_split_over_workgroups(lens):
    attend(lens, 1, 2, 64, 64, "f16", 11)
    attend(lens, 1, 2, 64, 64, "f16", 12, window=3000, prefix=[100] * len(lens))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("scores", ["rising", "falling", "one"])
@pytest.mark.parametrize("values", ["rising", "falling", "last", "small"])
def test_sizes_that_change_along_a_sequence(values, scores, kind):
    """Scores and values that grow or fall along the keys, so that maxima and the values' range move all the way."""
    rng = np.random.default_rng(27)
    heads, group, d, page, n = 2, 1, 64, 32, 700
    for queries in (1, 40):
        j = np.arange(n) / (n - 1)
        up = {"rising": j * 12 - 6, "falling": 6 - 12 * j, "last": np.where(np.arange(n) == n - 1, 13.0, -3.0),
              "small": np.full(n, -13.0)}[values]
        q = draw(rng, (queries, heads, d), kind, 0.1)
        along = q[0, 0] / np.abs(q[0, 0]).max()
        lean = {"rising": 40 * j - 20, "falling": 20 - 40 * j, "one": np.where(np.arange(n) == 333, 20.0, 0.0)}[scores]
        k = kv.round16(lean[:, None, None] * along * 0.3 + 0.2 * rng.standard_normal((n, heads, d)), kind)
        v = kv.round16(rng.standard_normal((n, heads, d)) * np.exp2(up)[:, None, None], kind)
        c = make_cache(-(-n // page), heads, d, page, kind)
        table = dev(np.arange(-(-n // page))[None], torch.int32)
        say(f"fp4_cache_attention with {values} values and {scores} scores, {queries} queries, {kind}")
        i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), torch.arange(n, device="cuda"))
        out, lse = i8.fp4_cache_attention(dev16(q, kind), c, table, dev(np.array([n]), torch.int32), max_q=queries,
                                          return_lse=True)
        torch.cuda.synchronize()
        check(out, lse, [(q, kv.dequantize(*kv.quantize(k)), kv.dequantize(*kv.quantize(v)))], d ** -0.5, kind)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_not_numbers_stay_where_they_are(kind):
    """A block of V that holds an infinity, at a key in sight: the other heads and blocks are as without it."""
    rng = np.random.default_rng(28)
    heads, d, page, n = 2, 128, 16, 90
    q, k, v = draw(rng, (3, heads, d), kind), draw(rng, (n, heads, d), kind, 0.3), draw(rng, (n, heads, d), kind)
    table = dev(np.arange(6)[None], torch.int32)
    outs = []
    say(f"fp4_cache_attention beside an infinity {kind}")
    for bad in (False, True):
        c = make_cache(6, heads, d, page, kind)
        if bad:
            v[40, 1, 70] = np.inf
        i8.fp4_cache_write(c, dev16(k, kind), dev16(v, kind), torch.arange(n, device="cuda"))
        outs.append(wide(i8.fp4_cache_attention(dev16(q, kind), c, table, dev(np.array([n]), torch.int32), max_q=3)))
    assert np.array_equal(outs[0][:, 0], outs[1][:, 0]) and np.array_equal(outs[0][:, 1, :64], outs[1][:, 1, :64])
    assert not np.isfinite(outs[1][:, 1, 64:]).any()


def test_strides_orders_and_out():
    """q and out as views (a fused projection's output, head-major), one kv head of a query count that is odd."""
    lens, heads, group, d = [(3, 50), (5, 33)], 2, 3, 128
    c, table, lengths, seqs = build(lens, heads, group, d, 32, "f16", 21)
    q = np.concatenate([s[0] for s in seqs])
    n, hq = q.shape[:2]
    qo = dev(np.array([0, 3, 8]), torch.int32)
    wide_q = torch.zeros((n, 2 * hq, d), dtype=torch.float16, device="cuda")
    wide_q[:, hq:] = dev16(q, "f16")
    head_major = dev16(q, "f16").transpose(0, 1).contiguous().transpose(0, 1)
    big = torch.full((n, hq + 4, d + 8), 9.0, dtype=torch.float16, device="cuda")
    table2 = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    table2[:, :table.shape[1]] = table
    say("fp4_cache_attention on views")
    a, la = i8.fp4_cache_attention(wide_q[:, hq:], c, table2[:, :table.shape[1]], lengths, qo, 5, return_lse=True)
    b = i8.fp4_cache_attention(head_major, c, table, lengths, qo, 5, out=big[:, 2:hq + 2, :d])
    torch.cuda.synchronize()
    check(a, la, seqs, d ** -0.5, "f16")
    assert torch.equal(a, b)
    big[:, 2:hq + 2, :d] = 9.0
    assert bool((big == 9.0).all())


@pytest.mark.parametrize("n", [1, 4, 70])
def test_pages_outside_the_cache_are_not_visible(n):
    lens, d, page = [(n, 100)], 64, 16
    c, table, lengths, seqs = build(lens, 1, 2, d, page, "f16", 22)
    bad = table.clone()
    bad[0, 1], bad[0, 4] = -5, 1 << 30
    hidden = np.zeros(100, bool)
    hidden[16:32] = hidden[64:80] = True
    say("fp4_cache_attention with page ids outside the cache")
    out, lse = i8.fp4_cache_attention(dev16(seqs[0][0], "f16"), c, bad, lengths, return_lse=True)
    gone = torch.full_like(bad, -1)
    out0, lse0 = i8.fp4_cache_attention(dev16(seqs[0][0], "f16"), c, gone, lengths, return_lse=True)
    torch.cuda.synchronize()
    check(out, lse, seqs, d ** -0.5, "f16", hidden=[hidden])
    assert bool((out0 == 0).all()) and bool(torch.isneginf(lse0).all())


def test_device_values_are_bounded():
    """Lengths past max_len and below 0, offsets past the rows of q, a sequence with more queries than max_q."""
    lens, d, page = [(2, 40), (2, 60)], 64, 16
    c, table, _, seqs = build(lens, 1, 1, d, page, "f16", 23)
    q = dev16(np.concatenate([s[0] for s in seqs]), "f16")
    say("fp4_cache_attention with lengths and offsets out of range")
    out, lse = i8.fp4_cache_attention(q, c, table, dev(np.array([1 << 30, -4]), torch.int32), max_q=2, max_len=40,
                                      return_lse=True)
    torch.cuda.synchronize()
    check(out[:2], lse[:2], seqs[:1], d ** -0.5, "f16")
    assert bool((out[2:] == 0).all()) and bool(torch.isneginf(lse[2:]).all())
    mark = torch.full_like(q, 5.0)
    out = i8.fp4_cache_attention(q, c, table, dev(np.array([40, 60]), torch.int32), dev(np.array([-3, 4, 900]), torch.int32),
                                 max_q=1, out=mark)
    torch.cuda.synchronize()
    assert bool((out[1:] == 5.0).all())                # one query a sequence at most, and no row past the last


def test_first_rows_do_not_depend_on_batch_or_padding():
    """A sequence's rows are the same numbers alone and in a batch, and twice in a row."""
    lens = [(1, 777), (1, 50), (1, 3000)]
    c, table, lengths, seqs = build(lens, 2, 4, 128, 64, "bf16", 24)
    q = dev16(np.concatenate([s[0] for s in seqs]), "bf16")
    say("fp4_cache_attention twice")
    a = i8.fp4_cache_attention(q, c, table, lengths, max_len=3000)
    b = i8.fp4_cache_attention(q, c, table, lengths, max_len=3000)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("lens", [[(1, 5000), (1, 40)], [(40, 300), (20, 20)]], ids=["decode", "prompt"])
def test_streams_graphs_and_workspace(lens):
    """On a side stream, into a graph that is replayed with eager work between, with a caller's workspace."""
    heads, group, d, page, kind = 2, 2, 128, 64, "f16"
    c, table, lengths, seqs = build(lens, heads, group, d, page, kind, 25)
    counts = [n for n, _ in lens]
    q = dev16(np.concatenate([s[0] for s in seqs]), kind)
    qo = dev(np.concatenate([[0], np.cumsum(counts)]), torch.int32)
    slots = dev(np.array([2 * page + 3]), torch.int64)
    k1, v1 = (dev16(draw(np.random.default_rng(i), (1, heads, d), kind), kind) for i in (1, 2))
    work = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")

    def step(out):
        i8.fp4_cache_write(c, k1, v1, slots)
        i8.fp4_cache_attention(q, c, table, lengths, qo, max(counts), out=out, workspace=work)

    say(f"fp4 cache step on a side stream and in a graph {lens}")
    eager = torch.empty_like(q)
    step(eager)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    side = torch.empty_like(q)
    with torch.cuda.stream(st):
        step(side)
    torch.cuda.synchronize()
    assert torch.equal(side, eager)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            step(out)
    torch.cuda.synchronize()
    for rep in range(4):
        out.fill_(1.0)
        work.fill_(rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), rep
        step(side)
        torch.cuda.synchronize()
        assert torch.equal(side, eager), rep


def test_empty_calls():
    c = make_cache(2, 1, 64, 16, "f16")
    before = c.data.clone()
    none = torch.empty((0, 1, 64), dtype=torch.float16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    say("fp4 cache: empty calls")
    i8.fp4_cache_write(c, none, none, slots)
    k, v = i8.fp4_cache_read(c, slots)
    assert k.shape == v.shape == (0, 1, 64)
    out = i8.fp4_cache_attention(none, c, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                                 torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 1, 64)
    q = torch.ones((2, 1, 64), dtype=torch.float16, device="cuda")
    out, lse = i8.fp4_cache_attention(q, c, torch.empty((2, 0), dtype=torch.int32, device="cuda"),
                                      torch.zeros(2, dtype=torch.int32, device="cuda"), return_lse=True)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all()) and torch.equal(before, c.data)


def test_refusals():
    c = make_cache(2, 2, 128, 16, "f16")
    f = dict(dtype=torch.float16, device="cuda")
    k = torch.zeros((3, 2, 128), **f)
    slots = torch.arange(3, device="cuda")
    with pytest.raises(TypeError):
        i8.fp4_cache_write(c, k.float(), k, slots)
    with pytest.raises(TypeError):
        i8.fp4_cache_write(c, k, k.to(torch.bfloat16), slots)
    with pytest.raises(ValueError):
        i8.fp4_cache_write(c, k[:, :1], k, slots)
    with pytest.raises(ValueError):
        i8.fp4_cache_write(c, k, k[:2], slots)
    with pytest.raises(ValueError):
        i8.fp4_cache_write(c, k, k, slots.int())
    with pytest.raises(ValueError):
        i8.fp4_cache_write(c, k, k, slots.cpu())
    with pytest.raises(ValueError):
        i8.fp4_cache_write(c, torch.zeros((3, 2, 256), **f)[:, :, ::2], k, slots)
    with pytest.raises(i8.I8mpError):                  # 16-byte alignment
        i8.fp4_cache_write(c, torch.zeros(3 * 2 * 128 + 8, **f)[1:769].view(3, 2, 128), k, slots)
    with pytest.raises(i8.I8mpError):                  # a token stride that is no multiple of 8
        i8.fp4_cache_write(c, torch.zeros((3, 260), **f)[:, :256].as_strided((3, 2, 128), (260, 128, 1)), k, slots)
    with pytest.raises(ValueError):
        i8.fp4_cache_read(c, slots, torch.int8)
    q, table, lengths = torch.zeros((2, 4, 128), **f), torch.zeros((2, 2), dtype=torch.int32, device="cuda"), \
        torch.ones(2, dtype=torch.int32, device="cuda")
    attend_ = i8.fp4_cache_attention
    assert attend_(q, c, table, lengths).shape == q.shape
    for bad in (dict(q=q.float()), dict(q=q[:, :, :64]), dict(table=table.long()), dict(table=table[:1]),
                dict(lengths=lengths.long()), dict(max_q=2), dict(alibi=torch.ones(3, device="cuda")),
                dict(prefix=torch.ones(1, dtype=torch.int32, device="cuda")),
                dict(q_offsets=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(out=q[:1]), dict(out=q.bfloat16()),
                dict(q=q.cpu())):
        args = dict(q=q, table=table, lengths=lengths)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            attend_(args.pop("q"), c, args.pop("table"), args.pop("lengths"), **args)
    for bad in (dict(q=torch.zeros((2, 3, 128), **f)), dict(window=-1), dict(softcap=-1.0), dict(softcap=float("nan")),
                dict(scale=float("inf")), dict(max_len=33), dict(max_len=-1),
                dict(q=torch.zeros(2 * 4 * 128 + 8, **f)[1:1025].view(2, 4, 128))):
        args = dict(q=q)
        args.update(bad)
        with pytest.raises(i8.I8mpError):
            attend_(args.pop("q"), c, table, lengths, **args)
    big = torch.zeros((1, 4, 128), **f)
    with pytest.raises(i8.I8mpError):                  # a workspace that is too small
        attend_(big, c, torch.zeros((1, 4096), dtype=torch.int32, device="cuda"), lengths[:1],
                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_prompts_that_fill_the_chip(kind):
    """Enough row tiles that each wave has one to itself: the rows of sampled heads and of all lengths' ends."""
    heads, group, d, page = 40, 1, 128, 64
    lens = [(500, 531), (420, 420), (511, 700), (333, 333), (480, 480), (470, 501), (509, 509), (390, 400), (1, 40)]
    c, table, lengths, seqs = build(lens, heads, group, d, page, kind, 29)
    counts = [n for n, _ in lens]
    assert (sum(counts) // 48 + len(lens)) * heads * 2 >= 2048 * 3
    q = dev16(np.concatenate([s[0] for s in seqs]), kind)
    qo = dev(np.concatenate([[0], np.cumsum(counts)]), torch.int32)
    say(f"fp4_cache_attention of {sum(counts)} queries, {heads} heads, {kind}")
    out, lse = i8.fp4_cache_attention(q, c, table, lengths, qo, max(counts), window=300, return_lse=True)
    torch.cuda.synchronize()
    few = [0, 17, 39]
    # rows near each sequence's start and end, as sequences that end there
    at = 0
    for (n, length), (qs, k, v) in zip(lens, seqs):
        for i in sorted({0, 1, 47, 48, n // 2, n - 2, n - 1}):
            if 0 <= i < n:
                end = length - n + i + 1
                check(out[at + i:at + i + 1, few], lse[at + i:at + i + 1, few],
                      [(qs[i:i + 1, few], k[:end, few], v[:end, few])], d ** -0.5, kind, window=300)
        at += n
