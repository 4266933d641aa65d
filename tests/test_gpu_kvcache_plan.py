"""Calls of every cut that the attention over the 4-bit cache makes, against the CPU
oracle at sampled rows, to the bounds of test_gpu_kvcache_edges.py.

Sequences share one store of tokens, each from a page of its own on, so that large
batches cost little; the values are those that the cache reads back, which other tests
pin to the oracle's."""

import numpy as np
import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from gpu_util import host, say
from oracle import kvcache as kv
from test_gpu_kvcache import DTYPE, dev, dev16, make_cache, wide
from test_gpu_kvcache_edges import check

pytestmark = pytest.mark.gpu


class Store:
    """Sequences lens = [(queries, length)] over shared tokens; table rows name shuffled pages.  Every 7th token from
    `small` on has values 2^-18 of the others'."""

    def __init__(self, lens, heads, group, d, page, kind, seed, extra_cols=0, small=None):
        rng = np.random.default_rng([72, seed])
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.heads, self.group, self.d, self.page, self.kind = lens, heads, group, d, page, kind
        self.first = [int(rng.integers(0, 6)) for _ in lens]                       # page that a sequence starts at
        pages = max(f - (-length // page) for f, (_, length) in zip(self.first, lens)) + 1
        ids = rng.permutation(pages)
        self.cols = max(max(-(-length // page) for _, length in lens), 1) + extra_cols
        table = np.full((len(lens), self.cols), -7)
        for i, (f, (_, length)) in enumerate(zip(self.first, lens)):
            used = -(-length // page)
            table[i, :used] = ids[f:f + used]
        self.cache = make_cache(pages, heads, d, page, kind, 0xFF)
        n = pages * page
        at = np.arange(n)
        slots = dev(ids[at // page] * page + at % page, torch.int64)
        k, v = (torch.randn((n, heads, d), generator=gen, device="cuda").to(DTYPE[kind]) for _ in range(2))
        if small is not None:
            v[small::7] *= 2.0 ** -9
            v[small + 1::7] *= 2.0 ** 9
        i8.fp4_cache_write(self.cache, k, v, slots)
        self.k, self.v = (wide(x) for x in i8.fp4_cache_read(self.cache, slots, torch.float32))
        self.table = dev(table, torch.int32)
        self.lengths = dev(np.array([length for _, length in lens]), torch.int32)
        self.counts = [c for c, _ in lens]
        self.offsets = np.concatenate([[0], np.cumsum(self.counts)])
        self.q = kv.round16(rng.standard_normal((int(self.offsets[-1]), heads * group, d), np.float32), kind)

    def run(self, rows=None, **kw):
        out, lse = i8.fp4_cache_attention(dev16(self.q, self.kind), self.cache, self.table, self.lengths,
                                          q_offsets=dev(self.offsets, torch.int32), max_q=max(self.counts), return_lse=True,
                                          **kw)
        torch.cuda.synchronize()
        return out, lse

    def compare(self, out, lse, picks, heads=None, **kw):
        """picks: (sequence, query) to compare; heads: kv heads (all of their query heads)."""
        heads = list(range(self.heads)) if heads is None else heads
        scale = kw.pop("scale", self.d ** -0.5)
        hq = [h * self.group + g for h in heads for g in range(self.group)]
        kw["prefix"] = None if kw.get("prefix") is None else host(kw["prefix"])
        if kw.get("alibi") is not None:
            kw["alibi"] = host(kw["alibi"])[hq]
        for b, i in picks:
            n, length = self.lens[b]
            at, row = self.first[b] * self.page, int(self.offsets[b]) + i
            more = dict(kw, prefix=None if kw["prefix"] is None else [int(kw["prefix"][b])])
            end = length - n + i + 1                       # tokens up to the query's own; a prefix may reach past it
            last = i == n - 1 or kw["prefix"] is None
            assert last, "a row with a prefix is compared as its sequence's last"
            end = max(end, 0)
            check(out[row:row + 1, hq], lse[row:row + 1, hq],
                  [(self.q[row:row + 1, hq], self.k[at:at + end, heads], self.v[at:at + end, heads])],
                  scale, self.kind, **more)


def test_a_prefix_longer_than_the_parts_allow_for():
    """Many segments under a short window: few parts each, which a long prefix makes long."""
    lens = [(1, 3000 + 37 * (i % 9)) for i in range(64)]
    lens[5], lens[20], lens[63] = (1, 0), (1, 17), (1, 3200)
    s = Store(lens, 8, 2, 64, 64, "f16", 1, extra_cols=500)
    prefix = np.full(64, 3)
    prefix[[0, 5, 7, 20, 40, 63]] = [2900, 40, 5000, 9, 1500, 100]
    say("fp4_cache_attention with long prefixes beside a window")
    kw = dict(window=64, prefix=dev(prefix, torch.int32))
    s.compare(*s.run(**kw), picks=[(b, 0) for b in (0, 1, 5, 7, 20, 40, 62, 63)], heads=[0, 7], **kw)
    kw = dict(window=64, prefix=dev(prefix[:1], torch.int32))
    s = Store([(3, 9001)], 2, 4, 128, 32, "bf16", 2, extra_cols=3000)
    s.compare(*s.run(**kw), picks=[(0, 2)], **kw)


def alibi_of(n):
    return torch.exp2(-8.0 * torch.arange(1, n + 1, device="cuda") / n).float()


def forms(q_heads):
    """Every form of the scores."""
    return [dict(), dict(softcap=20.0), dict(alibi=alibi_of(q_heads)), dict(softcap=500.0, window=900)]


KINDS = ["f16", "bf16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 16), (128, 128), (256, 16), (256, 32)])
def test_cut_decode(d, page, kind):
    """Few long sequences of one query: parts and their join, in rows of one set, and of two and three (group 17 and 40)."""
    for group in (1, 8, 17, 40) if d < 256 else (4, 20):
        s = Store([(1, 9003), (1, 40), (1, 0), (1, 6500)], 2, group, d, page, kind, d + group)
        for kw in forms(2 * group):
            say(f"fp4_cache_attention cut, 2 x {group} heads of {d}, pages of {page} {kind} {list(kw)}")
            s.compare(*s.run(**kw), picks=[(0, 0), (1, 0), (2, 0), (3, 0)], heads=[1], **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,page", [(64, 64), (128, 16), (128, 64), (256, 64)])
def test_cut_queries(d, page, kind):
    """Tens of queries behind long contexts, ragged: cut row tiles of 16 to 48 rows, the last ones not full."""
    for lens, group in (([(9, 5003), (7, 6400), (1, 90)], 2), ([(40, 7000), (33, 300), (50, 50)], 1), ([(70, 8001)], 2)):
        s = Store(lens, 2, group, d, page, kind, d + len(lens))
        for kw in forms(2 * group):
            say(f"fp4_cache_attention cut, {lens}, 2 x {group} heads of {d}, pages of {page} {kind} {list(kw)}")
            picks = [(b, i) for b, (n, _) in enumerate(lens) for i in sorted({0, n // 2, n - 1})]
            s.compare(*s.run(**kw), picks=picks, heads=[0], **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 128)])
def test_cut_batches(d, page, kind):
    """512 segments of uneven lengths: the join in workgroups of many rows, parts of several tiles a wave."""
    lens = [(1, 5000 + 160 * i) for i in range(60)] + [(1, 1), (1, 0), (1, 4097), (1, 200)]
    s = Store(lens, 8, 2, d, page, kind, d + 1)
    for kw in forms(16)[:2]:
        say(f"fp4_cache_attention of 64 sequences cut, heads of {d} {kind} {list(kw)}")
        s.compare(*s.run(**kw), picks=[(b, 0) for b in (0, 31, 59, 60, 61, 62, 63)], heads=[0, 7], **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (128, 16), (256, 32)])
def test_whole_contexts_of_eight_and_four_waves(d, page, kind):
    for n, length in ((20, 900), (70, 1500)):
        lens = [(1, length - 13 * i) for i in range(n)]
        s = Store(lens, 4, 2, d, page, kind, d + n)
        for kw in forms(8):
            say(f"fp4_cache_attention of {n} whole contexts, heads of {d}, pages of {page} {kind} {list(kw)}")
            s.compare(*s.run(**kw), picks=[(0, 0), (n // 2, 0), (n - 1, 0)], heads=[3], **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 64])
def test_prompts_of_one_wave_each_behind_long_contexts(page, kind):
    """Row tiles that have a wave to themselves, with more than 64 tiles of keys: its list of pages is read again."""
    lens = [(1800, 4300), (1500, 3001)]
    s = Store(lens, 24, 2, 128, page, kind, 5)
    assert (3300 * 2 // 48 + 2) * 24 * 2 >= 2048 * 3
    for kw in forms(48) + [dict(window=2500), dict(prefix=dev(np.array([100, 3001]), torch.int32))]:
        say(f"fp4_cache_attention of prompts by single waves, pages of {page} {kind} {list(kw)}")
        last = [(0, 1799), (1, 1499)]
        s.compare(*s.run(**kw), picks=last + ([] if "prefix" in kw else [(0, 0), (0, 23), (0, 900), (1, 0), (1, 1490)]),
                  heads=[0, 23], **kw)


@pytest.mark.parametrize("kind", KINDS)
def test_prompts_of_four_waves_behind_long_contexts(kind):
    """Whole contexts of more than 256 tiles: the list of pages is read again with four waves too."""
    lens = [(2400, 9100), (2300, 10007), (2350, 8800), (2400, 9999)]
    s = Store(lens, 16, 1, 64, 32, kind, 6)
    say(f"fp4_cache_attention of prompts behind long contexts {kind}")
    s.compare(*s.run(), picks=[(0, 0), (0, 2399), (1, 1200), (1, 2299), (2, 47), (3, 48), (3, 2399)], heads=[0, 15])


@pytest.mark.parametrize("d,page,group", [(64, 16, 1), (64, 64, 40), (128, 16, 20), (128, 64, 1), (256, 16, 4), (256, 64, 1)])
@pytest.mark.parametrize("small", [0, 2300])
def test_wide_values_in_every_plan(d, page, group, small):
    """fp16 values whose sizes span 2^18 from the first key on, or only from one far behind: cut, whole, prompts."""
    for lens in ([(1, 9003), (1, 50)], [(1, 900 + i) for i in range(20)], [(30, 3001), (50, 2400)], [(3, 2330)]):
        s = Store(lens, 2, group, d, page, "f16", d + len(lens), small=small if lens[0][1] > 2300 else 0)
        for kw in forms(2 * group)[:2]:
            say(f"fp4_cache_attention of wide values from {small}, {lens[:2]}, 2 x {group} heads of {d} {list(kw)}")
            n = lens[0][0]
            picks = [(0, 0), (0, n - 1), (len(lens) - 1, lens[-1][0] - 1)]
            s.compare(*s.run(**kw), picks=picks, heads=[1], **kw)


@pytest.mark.parametrize("small", [0, 2300])
def test_wide_values_by_single_waves(small):
    s = Store([(1800, 4300), (1500, 3001)], 24, 2, 128, 64, "f16", 7, small=small)
    for kw in forms(48):
        say(f"fp4_cache_attention of prompts by single waves, wide values from {small} {list(kw)}")
        s.compare(*s.run(**kw), picks=[(0, 0), (0, 23), (0, 1799), (1, 700), (1, 1499)], heads=[11], **kw)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_are_the_same_alone_and_in_a_batch(kind):
    """Whole contexts, which take eight waves alone and in the batch."""
    lens = [(1, 777), (1, 50), (1, 700), (1, 333)]
    s = Store(lens, 2, 4, 128, 64, kind, 8)
    q = dev16(s.q, kind)
    say(f"fp4_cache_attention alone and in a batch {kind}")
    out, lse = s.run(max_len=800)
    s.compare(out, lse, picks=[(b, 0) for b in range(4)])
    for b in range(4):
        one, one_lse = i8.fp4_cache_attention(q[b:b + 1], s.cache, s.table[b:b + 1], s.lengths[b:b + 1], max_len=800,
                                              return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(one[0], out[b]) and torch.equal(one_lse[0], lse[b])
    again, _ = s.run(max_len=800)
    assert torch.equal(again, out)


@pytest.mark.parametrize("kind", KINDS)
def test_far_caps_beside_the_other_terms(kind):
    s = Store([(1, 700), (5, 333), (38, 90)], 2, 2, 128, 16, kind, 9)
    pre = dev(np.array([40, 0, 1000]), torch.int32)
    for cap in (65.0, 400.0):
        for scale in (0.3, -0.3):
            for more in (dict(alibi=alibi_of(4)), dict(prefix=pre, window=20), dict(alibi=alibi_of(4), prefix=pre)):
                kw = dict(more, softcap=cap, scale=scale)
                say(f"fp4_cache_attention capped at {cap}, factor {scale}, {list(more)} {kind}")
                s.compare(*s.run(**kw), picks=[(0, 0), (1, 4), (2, 37)], **kw)
