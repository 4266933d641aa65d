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
from test_gpu_kvcache import DTYPE, dev, dev16, draw, make_cache, wide
from test_gpu_kvcache_edges import check

pytestmark = pytest.mark.gpu


class Store:
    """Sequences lens = [(queries, length)] over shared tokens; table rows name shuffled pages."""

    def __init__(self, lens, heads, group, d, page, kind, seed, extra_cols=0):
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
        i8.fp4_cache_write(self.cache, k, v, slots)
        self.k, self.v = (wide(x) for x in i8.fp4_cache_read(self.cache, slots, torch.float32))
        self.table = dev(table, torch.int32)
        self.lengths = dev(np.array([length for _, length in lens]), torch.int32)
        self.counts = [c for c, _ in lens]
        self.offsets = np.concatenate([[0], np.cumsum(self.counts)])
        self.q = draw(rng, (int(self.offsets[-1]), heads * group, d), kind, 0.3)

    def run(self, rows=None, **kw):
        out, lse = i8.fp4_cache_attention(dev16(self.q, self.kind), self.cache, self.table, self.lengths,
                                          q_offsets=dev(self.offsets, torch.int32), max_q=max(self.counts), return_lse=True,
                                          **kw)
        torch.cuda.synchronize()
        return out, lse

    def compare(self, out, lse, picks, heads=None, **kw):
        """picks: (sequence, query) to compare; heads: kv heads (all of their query heads)."""
        heads = list(range(self.heads)) if heads is None else heads
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
                  self.d ** -0.5, self.kind, **more)


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
