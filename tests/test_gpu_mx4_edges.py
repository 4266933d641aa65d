"""Microscaled calls at the borders between their kernels, and two of them at once.

Rows so long that the streaming kernel's LDS holds few of them, gradients with so few
rows that they take that kernel, calls on two streams.  Bounds as in test_gpu_mx4.py."""

import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
import test_gpu_mx4 as base
from gpu_util import say

pytestmark = pytest.mark.gpu

DTYPE, STEP = base.DTYPE, base.STEP


def back(t, columns=False):
    return i8.mx4_dequantize(i8.mx4_quantize(t, columns), torch.float32).double()


def close(got, a, b, kind):
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    kp = -(-a.shape[1] // 128) * 128
    tol = (kp / 64 + 64) * 2.0 ** -23 * size + torch.finfo(DTYPE[kind]).eps / 2 * want.abs() + STEP[kind]
    assert got.shape == want.shape and bool(((got.double() - want).abs() <= tol).all())


# 64 KiB hold 64, 15, 6 and 4 rows of scales; one element more and tiles take over
@pytest.mark.parametrize("case", [(16, 300, 30000), (5, 70, 131072), (16, 33, 300000), (3, 21, 524032), (3, 21, 524033), (1, 5, 1 << 21)],
                         ids=lambda c: "%dx%dx%d" % c)
def test_long_rows(case):
    base.test_matmul_exact_sums_large(case)


# the last k at which x is quantized beside the weights, and the next
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 99584), (1, 99585), (2, 53000), (4, 28928), (4, 28929), (3, 41), (5, 28928)])
def test_linear_of_long_rows(m, k, kind):
    n = 75
    gen = torch.Generator(device="cuda").manual_seed(k)
    x, w = (torch.randn((r, k + 1), generator=gen, device="cuda").to(DTYPE[kind])[:, 1:] for r in (m, n))
    bias = torch.zeros(n, dtype=DTYPE[kind], device="cuda")
    say(f"mx4_linear long rows {m} {k} {kind}")
    got = i8.mx4_linear(x, i8.mx4_quantize(w), bias)
    close(got, back(x), back(w), kind)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("case", [(300, 7, 500), (2000, 16, 24), (5, 300, 9), (16, 1000, 16), (17, 17, 17), (4000, 1, 130), (1, 4000, 1)],
                         ids=lambda c: "%dx%dx%d" % c)
def test_gradients_of_few_rows(case, kind):
    m, n, k = case
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    g, x, w = (torch.randn(s, generator=gen, device="cuda").to(DTYPE[kind]) for s in ((m, n), (m, k), (n, k)))
    say(f"mx4_linear_backward few rows {case} {kind}")
    gx, gw = i8.mx4_linear_backward(g, x, w)
    close(gx, back(g), back(w, True), kind)
    close(gw, back(g, True), back(x, True), kind)


def test_two_calls_at_once():
    """Calls on two streams, each with memory of its own, give what they give alone."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").half()
    work = []
    for m, n, k in ((100, 300, 9000), (3, 5000, 4096), (700, 900, 1000), (16, 600, 20000)):
        x, w, g = rand(m, k), rand(n, k), rand(m, n)
        q = i8.mx4_quantize(w)
        work.append(lambda x=x, q=q: (i8.mx4_linear(x, q),))
        work.append(lambda x=x, w=w, g=g: i8.mx4_linear_backward(g, x, w))
    t = rand(500, 12, 128)
    slots, where = torch.randperm(512, generator=gen, device="cuda")[:500], torch.arange(500, device="cuda")
    angle = torch.rand((500, 64), generator=gen, device="cuda")
    caches = [i8.Fp4Cache.create(8, 4, 128) for _ in range(3)]
    append = lambda c: i8.fp4_cache_append(c, t[:, :4], t[:, 4:8], t[:, 8:], slots, where, angle.cos(), angle.sin())
    say("mx4 two calls at once")
    want = [f() for f in work]
    turned = append(caches[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(5):
        got = [[], []]
        for i in range(len(work)):
            for s, stream in enumerate(streams):
                with torch.cuda.stream(stream):
                    j = i if s == 0 else len(work) - 1 - i
                    got[s].append((j, work[j]()))
                    if i == turn:
                        got[s].append((None, append(caches[s])))
        torch.cuda.synchronize()
        for s in range(2):
            for j, out in got[s]:
                if j is None:
                    assert torch.equal(out, turned) and torch.equal(caches[s].data, caches[2].data)
                else:
                    assert all(torch.equal(a, b) for a, b in zip(out, want[j]))
        for c in caches[:2]:
            c.data.zero_()
