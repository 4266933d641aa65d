"""GPU parity of the append to the 4-bit cache: keys and queries rotated by position.

Bit-exact: the rotation is defined as the exact value rounded to fp32, then to the
16-bit type (float64 stands for the exact value on both sides), and the cache holds what
fp4_cache_write of the keys so rotated leaves, byte for byte."""

import numpy as np
import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from gpu_util import host, say
from oracle import mx4
from oracle.kvcache import round16

pytestmark = pytest.mark.gpu

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
BITS = torch.int16


def dev16(x, kind):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(DTYPE[kind])


def turned(x, cos, sin, inter, kind):
    y = mx4.rotate(x.astype(np.float64), cos, sin, inter).astype(np.float32)
    return dev16(round16(y, kind), kind)


def tables(rows, half):
    rate = np.exp2(-np.arange(half) / half * 13.0)
    angle = np.arange(rows)[:, None] * rate
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


CASES = [
    # tokens, q heads, kv heads, head_dim, rotary, page, pages, type
    (1, 1, 1, 64, 64, 16, 1, "f16"),
    (1, 40, 40, 128, 128, 64, 2, "f16"),
    (3, 6, 2, 256, 256, 32, 2, "bf16"),
    (17, 9, 3, 128, 64, 16, 5, "bf16"),
    (65, 4, 2, 64, 16, 256, 2, "f16"),
    (200, 7, 1, 128, 96, 128, 3, "f16"),
    (333, 1, 1, 256, 112, 64, 7, "bf16"),
    (40, 5, 5, 64, 48, 16, 4, "bf16"),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("order", ["run", "scattered"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "t%d_q%d_k%d_d%d_r%d_p%d_x%d_%s" % c)
def test_append_bit_exact(case, order, inter):
    n, heads, kv, d, rotary, page, pages, kind = case
    rng = np.random.default_rng([90, n, heads, d])
    x = round16((rng.standard_normal((n, heads + 2 * kv, d)) * np.exp(rng.standard_normal((n, 1, 1)))).astype(np.float32), kind)
    x[0, heads, :16] = 0
    x[0, 0, 1] = -0.0
    cos, sin = tables(n + 9, rotary // 2)
    slots = rng.permutation(pages * page)[:n] if order == "scattered" else np.arange(n) + (pages * page - n) // 2
    where = rng.permutation(n + 9)[:n] if order == "scattered" else np.arange(n) + 3
    if n > 10:
        slots[3], slots[7], slots[9] = -1, pages * page, 1 << 40
        where[3], where[5] = -7, 1 << 40                             # taken into the tables
    row = np.clip(where, 0, n + 8)
    t = dev16(x, kind)
    q, k, v = t[:, :heads], t[:, heads:heads + kv], t[:, heads + kv:]
    ts, tp = torch.from_numpy(slots).cuda(), torch.from_numpy(where).cuda()
    tc, tn = (torch.from_numpy(np.pad(a, ((0, 0), (1, 2)))).cuda()[:, 1:1 + rotary // 2] for a in (cos, sin))
    one, two = (i8.Fp4Cache.create(pages, kv, d, page, DTYPE[kind]) for _ in range(2))
    one.data.fill_(0xA5)
    two.data.fill_(0xA5)
    say(f"fp4_cache_append {case} {order} {inter}")
    got = i8.fp4_cache_append(one, q, k, v, ts, tp, tc, tn, interleaved=inter)
    wq = turned(x[:, :heads], cos[row], sin[row], inter, kind)
    wk = turned(x[:, heads:heads + kv], cos[row], sin[row], inter, kind)
    assert torch.equal(got.view(BITS), wq.view(BITS))
    i8.fp4_cache_write(two, wk, v, ts)
    assert torch.equal(one.data, two.data)
    # without queries, and in place in the projection's output
    one.data.fill_(0xA5)
    assert i8.fp4_cache_append(one, None, k, v, ts, tp, tc, tn, inter) is None
    assert torch.equal(one.data, two.data)
    one.data.fill_(0xA5)
    assert i8.fp4_cache_append(one, q, k, v, ts, tp, tc, tn, inter, out=q) is q
    assert torch.equal(q.contiguous().view(BITS), wq.view(BITS)) and torch.equal(one.data, two.data)
    assert torch.equal(t[:, heads:].contiguous().view(BITS), dev16(x[:, heads:], kind).view(BITS))


def test_values_that_are_no_numbers():
    """A NaN or an infinity turns its pair alone, and is written as fp4_cache_write writes it."""
    rng = np.random.default_rng(91)
    x = round16(rng.standard_normal((4, 3, 64)).astype(np.float32), "f16")
    x[1, 0, 5], x[2, 1, 40] = np.nan, np.inf
    cos, sin = tables(4, 32)
    t = dev16(x, "f16")
    slots = torch.arange(4, device="cuda")
    tc, tn = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    one, two = (i8.Fp4Cache.create(1, 1, 64, 16) for _ in range(2))
    say("fp4_cache_append nan")
    got = i8.fp4_cache_append(one, t[:, :1], t[:, 1:2], t[:, 2:], slots, slots, tc, tn)
    bad = torch.isnan(got).nonzero().tolist()
    assert bad == [[1, 0, 5], [1, 0, 37]]
    k = torch.where(torch.isnan(t[:, 1:2]), 0, t[:, 1:2])
    k = turned(host(k.float()), cos, sin, False, "f16")
    i8.fp4_cache_write(two, k, t[:, 2:], slots)
    assert torch.equal(one.data, two.data)


def test_streams_graphs_and_refusals():
    rng = np.random.default_rng(92)
    x = [dev16(round16(rng.standard_normal((20, 8, 128)).astype(np.float32), "bf16"), "bf16") for _ in range(3)]
    cos, sin = (torch.from_numpy(a).cuda() for a in tables(64, 64))
    slots, where = torch.randperm(64, device="cuda")[:20], torch.arange(20, device="cuda") + 30
    one, two = (i8.Fp4Cache.create(4, 2, 128, 16, torch.bfloat16) for _ in range(2))
    say("fp4_cache_append graph")
    cur, stream, graph = x[0].clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    run = lambda c, t: i8.fp4_cache_append(c, t[:, :4], t[:, 4:6], t[:, 6:], slots, where, cos, sin)
    want = run(two, cur)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            got = run(one, cur)
    torch.cuda.synchronize()
    for t in x:
        cur.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = run(two, t)
        assert torch.equal(got, want) and torch.equal(one.data, two.data)
    t = x[0]
    q, k, v = t[:, :4], t[:, 4:6], t[:, 6:]
    for f, error in ((lambda: i8.fp4_cache_append(one, q, k, v, slots[:19], where, cos, sin), ValueError),
                     (lambda: i8.fp4_cache_append(one, q, k, v, slots, where.int(), cos, sin), ValueError),
                     (lambda: i8.fp4_cache_append(one, q, k, v, slots, where, cos[:, :-8], sin), ValueError),
                     (lambda: i8.fp4_cache_append(one, q, k, v, slots, where, cos[:0], sin[:0]), ValueError),
                     (lambda: i8.fp4_cache_append(one, q, k, v, slots, where, cos.double(), sin.double()), TypeError),
                     (lambda: i8.fp4_cache_append(one, q, k, v, slots, where, cos[:, :4], sin[:, :4]), i8.I8mpError),
                     (lambda: i8.fp4_cache_append(one, q[:19], k, v, slots, where, cos, sin), ValueError),
                     (lambda: i8.fp4_cache_append(one, None, k, v, slots, where, cos, sin, out=q), ValueError),
                     (lambda: i8.fp4_cache_append(one, q, k, v, slots, where, cos, sin, out=k), ValueError),
                     (lambda: i8.fp4_cache_append(one, q.half(), k, v, slots, where, cos, sin), TypeError),
                     (lambda: i8.fp4_cache_append(one, q, k, v[:, :1], slots, where, cos, sin), ValueError)):
        with pytest.raises(error):
            f()
    empty = i8.fp4_cache_append(one, q[:0], k[:0], v[:0], slots[:0], where[:0], cos, sin)
    assert empty.shape == (0, 4, 128)
