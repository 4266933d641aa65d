"""Calls that are cut into several launches give what one launch gives, bit for bit.

Moves of the 4-bit cache and the microscaled quantization are cut by workgroups: the
library's limit is lowered here, so that small calls are cut.  Dequantization is cut by
the rows of a grid, and one append is long enough for the limit as it is."""

import ctypes

import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from gpu_util import say

pytestmark = pytest.mark.gpu

BITS = torch.int16


@pytest.fixture
def limit():
    at = ctypes.c_int64.in_dll(i8.lib(), "i8mp_launch_blocks")
    whole = at.value
    assert whole == 1 << 22

    def lower(n):
        at.value = n

    yield lower
    at.value = whole


def same(a, b):
    return torch.equal(a.contiguous().view(BITS), b.contiguous().view(BITS))


def angles(gen, rows, half):
    a = torch.rand((rows, half), generator=gen, device="cuda") * 6.28
    return a.cos(), a.sin()


# tokens, q heads, kv heads, head_dim, launch's workgroups: pieces by the cache's lanes, by q's, and of one span
MOVES = [(3001, 3, 2, 64, 64), (3001, 40, 2, 128, 64), (700, 9, 9, 256, 20), (700, 33, 1, 64, 1), (65, 1, 1, 128, 1)]


@pytest.mark.parametrize("order", ["run", "scattered"])
@pytest.mark.parametrize("case", MOVES, ids=lambda c: "t%d_q%d_k%d_d%d_at%d" % c)
def test_cache_moves(case, order, limit):
    n, heads, kv, d, most = case
    gen = torch.Generator(device="cuda").manual_seed(n + heads)
    t = torch.randn((n, heads + 2 * kv, d), generator=gen, device="cuda").half()
    q, k, v = t[:, :heads], t[:, heads:heads + kv], t[:, heads + kv:]
    pages = -(-n // 32) + 2
    slots = torch.randperm(pages * 32, generator=gen, device="cuda")[:n] if order == "scattered" else torch.arange(n, device="cuda") + 5
    slots[n // 2] = -1
    where = torch.randint(0, 99, (n,), generator=gen, device="cuda")
    cos, sin = angles(gen, 99, d // 4)
    one, two = (i8.Fp4Cache.create(pages, kv, d, 32) for _ in range(2))
    for cache in (one, two):
        cache.data.fill_(0xA5)
    want = i8.fp4_cache_append(one, q, k, v, slots, where, cos, sin)
    wk, wv = i8.fp4_cache_read(one, slots)
    say(f"cut cache moves {case} {order}")
    limit(most)
    got = i8.fp4_cache_append(two, q, k, v, slots, where, cos, sin)
    assert same(got, want) and torch.equal(one.data, two.data)
    rk, rv = i8.fp4_cache_read(two, slots)
    assert same(rk, wk) and same(rv, wv)
    two.data.fill_(0xA5)
    i8.fp4_cache_write(two, k, v, slots)
    limit(1 << 22)
    one.data.fill_(0xA5)
    i8.fp4_cache_write(one, k, v, slots)
    assert torch.equal(one.data, two.data)
    limit(most)
    assert i8.fp4_cache_append(two, q, k, v, slots, where, cos, sin, out=q) is q and same(q, want)


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("m,k,left,most", [(1000, 300, 0, 16), (1111, 700, 1, 16), (4099, 40, 3, 4), (257, 2049, 2, 1), (130, 5000, 0, 8)])
def test_quantize(m, k, left, most, columns, limit):
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn((m, k + 5), generator=gen, device="cuda").half()[:, left:left + k]
    x[m // 2, 3], x[m - 1, k - 1] = float("nan"), float("inf")
    rows, length = (k, m) if columns else (m, k)
    kp = -(-length // 128) * 128
    want = i8.mx4_quantize(x, columns)
    wide = [torch.full((rows + 1, kp // 2 + 16), 0xA5, dtype=torch.uint8, device="cuda"),
            torch.full((rows + 1, kp // 32 + 4), 0xA5, dtype=torch.uint8, device="cuda")]
    say(f"cut mx4_quantize {m} {k} {left} columns={columns}")
    limit(most)
    got = i8.mx4_quantize(x, columns, i8.Mx4Tensor(wide[0][:rows], wide[1][:rows], length))
    for t, part, used in ((want.codes, wide[0], kp // 2), (want.scales, wide[1], kp // 32)):
        assert torch.equal(part[:rows, :used], t)
        assert bool((part[rows:] == 0xA5).all()) and bool((part[:, used:] == 0xA5).all())
    assert got.shape == (rows, length)


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n,k,most", [(3000, 2901, 200, 64), (2701, 3200, 136, 24), (300, 400, 500, 16)])
def test_backward(m, n, k, most, kind, limit):
    """The larger ones quantize grad_out by rows and by columns at once."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    g, x, w = (torch.randn(s, generator=gen, device="cuda").to(kind) for s in ((m, n), (m, k), (n, k)))
    want = i8.mx4_linear_backward(g, x, w)
    say(f"cut mx4_linear_backward {m} {n} {k} {kind}")
    limit(most)
    got = i8.mx4_linear_backward(g, x, w)
    assert same(got[0], want[0]) and same(got[1], want[1])


@pytest.mark.parametrize("kind", [torch.float16, torch.float32])
def test_dequantize_of_more_rows_than_a_grid_has(kind):
    """64 rows a workgroup, 65535 workgroups a launch."""
    cut = 64 * 65535
    rows, k = cut + 200, 7
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((rows, k), generator=gen, device="cuda").half()
    say(f"cut mx4_dequantize {kind}")
    q = i8.mx4_quantize(x)
    wide = torch.full((rows, k + 2), 7.0, dtype=kind, device="cuda")
    i8.mx4_dequantize(q, kind, wide[:, 1:1 + k])
    for a, b in ((0, 300), (cut - 300, cut + 200)):
        part = i8.Mx4Tensor(q.codes[a:b], q.scales[a:b], k)
        assert torch.equal(wide[a:b, 1:1 + k], i8.mx4_dequantize(part, kind))
        again = i8.mx4_quantize(x[a:b])
        assert torch.equal(again.codes, part.codes) and torch.equal(again.scales, part.scales)
    assert bool((wide[:, 0] == 7).all()) and bool((wide[:, 1 + k] == 7).all())


def test_an_append_of_more_tokens_than_a_launch_takes():
    """2^22 workgroups, nine a span of 32 tokens: two launches, the second of a few tokens."""
    cut = (1 << 22) // 9 * 32
    n, d = cut + 100, 64
    gen = torch.Generator(device="cuda").manual_seed(4)
    t = torch.zeros((n, 4, d), dtype=torch.float16, device="cuda")
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    where = torch.zeros(n, dtype=torch.int64, device="cuda")
    cos, sin = angles(gen, 50, d // 2)
    near = slice(cut - 100, n)
    t[near] = torch.randn((200, 4, d), generator=gen, device="cuda").half()
    slots[near] = torch.arange(200, device="cuda") + 3
    where[near] = torch.randint(0, 50, (200,), generator=gen, device="cuda")
    one, two = (i8.Fp4Cache.create(8, 1, d, 32) for _ in range(2))
    split = lambda x: (x[:, :2], x[:, 2:3], x[:, 3:])
    say("cut fp4_cache_append at size")
    want = i8.fp4_cache_append(one, *split(t[near]), slots[near], where[near], cos, sin)
    q = split(t)[0]
    assert i8.fp4_cache_append(two, *split(t), slots, where, cos, sin, out=q) is q
    assert same(q[near], want) and torch.equal(one.data, two.data) and not bool(q[:cut - 100].any())
