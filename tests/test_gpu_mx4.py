"""GPU parity of the microscaled 4-bit matrices against the CPU oracle.

Bit-exact: codes, scales and their padding, what is dequantized, and products whose sums
are whole quarters below 2^22 (every order of fp32 additions gives them).

Other products, element by element: terms are exact, a sum over k runs through at most
kp / 64 + 64 fp32 additions in any split, each off by at most 2^-23 of the sum of
magnitudes S (the matrix instruction's own additions among them), so
  |out - oracle| <= (kp / 64 + 64) 2^-23 S + u |oracle| + t
with u = eps / 2 of out's type and t half its smallest step.
"""

import numpy as np
import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from gpu_util import host, say
from oracle import mx4
from oracle.kvcache import round16

pytestmark = pytest.mark.gpu

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
STEP = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}


def wide(t):
    return host(t.double())


def dev16(x, kind):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(DTYPE[kind])


def rand16(rng, shape, kind, spread=0.0):
    return round16((rng.standard_normal(shape) * np.exp(rng.standard_normal(shape) * spread)).astype(np.float32), kind)


def held(codes, scales, k, extra=(0, 0)):
    """The Mx4Tensor of one-byte codes [rows, kp] and scale bytes, with rows that are longer by `extra` bytes."""
    c, s = mx4.pack(codes), np.asarray(scales, np.uint8)
    out = []
    for x, more in ((c, extra[0]), (s, extra[1])):
        t = torch.full((x.shape[0], x.shape[1] + more), 0xFF, dtype=torch.uint8, device="cuda")
        t[:, :x.shape[1]] = torch.from_numpy(x).cuda()
        out.append(t)
    return i8.Mx4Tensor(*out, k)


def drawn(rng, rows, k, low=127, high=128):
    """Random codes and scales in [low, high), padding zero."""
    kp = -(-k // 128) * 128
    codes = rng.integers(0, 16, (rows, kp)).astype(np.uint8)
    codes[:, k:] = 0
    return codes, rng.integers(low, high, (rows, kp // 32)).astype(np.uint8)


def close(got, want, size, kp, kind, extra=0.0):
    tol = (kp / 64 + 64) * 2.0 ** -23 * size + torch.finfo(DTYPE[kind]).eps / 2 * np.abs(want) + STEP[kind] + extra
    err = np.abs(wide(got) - want)
    assert err.shape == tol.shape and np.all(err <= tol), (np.argwhere(~(err <= tol))[:3], np.nanmax(err / tol))


# ---- quantization -----------------------------------------------------------------

SHAPES = [(1, 1), (1, 32), (3, 33), (7, 127), (5, 128), (2, 129), (64, 255), (33, 1000), (1, 5120), (300, 513), (1025, 96), (17, 2049)]


def check_quantized(q, x):
    codes, scales = mx4.quantize(x)
    assert np.array_equal(host(q.codes), mx4.pack(codes))
    assert np.array_equal(host(q.scales), scales)
    return codes, scales


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
@pytest.mark.parametrize("columns", [False, True])
def test_quantize_bit_exact(shape, kind, columns):
    rng = np.random.default_rng([80, *shape])
    x = rand16(rng, shape, kind, 2.0)
    x[shape[0] // 2] = 0
    x[0, 0] = -0.0
    say(f"mx4_quantize {shape} {kind} columns={columns}")
    q = i8.mx4_quantize(dev16(x, kind), columns)
    assert q.shape == (shape[::-1] if columns else shape)
    codes, scales = check_quantized(q, x.T if columns else x)
    v = mx4.values(codes, scales)[:, :q.k]
    for name, t in DTYPE.items():
        assert torch.equal(i8.mx4_dequantize(q, t).cpu(), torch.from_numpy(v).to(t)), name


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_quantize_every_16_bit_value(kind, columns):
    """Every pattern in blocks of neighbouring and of random magnitudes, NaNs and infinities among them."""
    rng = np.random.default_rng(81)
    order = [np.arange(65536), rng.permutation(65536), np.arange(65536).reshape(2048, 32).T.reshape(-1)]
    bits = np.concatenate(order).astype(np.uint16).reshape(-1, 4096)
    t = torch.from_numpy(bits.view(np.int16)).cuda().view(DTYPE[kind])
    say(f"mx4_quantize all {kind} columns={columns}")
    q = i8.mx4_quantize(t.t().contiguous() if columns else t, columns)
    check_quantized(q, wide(t))
    got = i8.mx4_dequantize(q, torch.float32)
    want = torch.from_numpy(mx4.values(*mx4.quantize(wide(t)))).float()
    assert torch.equal(torch.nan_to_num(got.cpu(), 7.0, 8.0, 9.0), torch.nan_to_num(want, 7.0, 8.0, 9.0))


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("left,right", [(1, 0), (8, 3), (3, 5)])
def test_quantize_views(left, right, columns):
    """Columns of a wider matrix, at any alignment, into rows that are longer than they need be."""
    rng = np.random.default_rng([82, left])
    x = rand16(rng, (70, 300 + left + right), "f16", 1.0)
    view = dev16(x, "f16")[:, left:left + 300]
    rows, k = (300, 70) if columns else (70, 300)
    kp = -(-k // 128) * 128
    big = i8.Mx4Tensor(torch.full((rows + 1, kp // 2 + 32), 0xA5, dtype=torch.uint8, device="cuda"),
                       torch.full((rows + 1, kp // 32 + 8), 0xA5, dtype=torch.uint8, device="cuda"), k)
    out = i8.Mx4Tensor(big.codes[:rows], big.scales[:rows], k)
    say(f"mx4_quantize view {left} {right} columns={columns}")
    assert i8.mx4_quantize(view, columns, out) is out
    want = x[:, left:left + 300]
    codes, scales = mx4.quantize(want.T if columns else want)
    assert np.array_equal(host(out.codes[:, :kp // 2]), mx4.pack(codes)) and np.array_equal(host(out.scales[:, :kp // 32]), scales)
    for t, used in ((big.codes, kp // 2), (big.scales, kp // 32)):
        assert bool((t[:, used:] == 0xA5).all()) and bool((t[rows:] == 0xA5).all())
    wider = torch.full((rows, k + 5), 3.0, dtype=torch.float16, device="cuda")
    i8.mx4_dequantize(out, out=wider[:, 2:2 + k])
    assert np.array_equal(wide(wider[:, 2:2 + k]), mx4.values(codes, scales)[:, :k])
    assert bool((wider[:, :2] == 3).all()) and bool((wider[:, 2 + k:] == 3).all())


def test_empty_calls():
    say("mx4 empty")
    for m, k in ((0, 64), (5, 0), (0, 0)):
        x = torch.zeros((m, k), dtype=torch.float16, device="cuda")
        for columns in (False, True):
            q = i8.mx4_quantize(x, columns)
            assert q.shape == ((k, m) if columns else (m, k)) and i8.mx4_dequantize(q).shape == q.shape
    bias = torch.arange(6, dtype=torch.float32, device="cuda")
    e = i8.mx4_quantize(torch.zeros((5, 0), dtype=torch.float16, device="cuda"))
    f = i8.mx4_quantize(torch.zeros((6, 0), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(i8.mx4_matmul(e, f, bias, torch.float32), bias.expand(5, 6))
    assert not i8.mx4_matmul(e, f).any()
    assert i8.mx4_matmul(i8.Mx4Tensor.create(0, 100), i8.Mx4Tensor.create(6, 100)).shape == (0, 6)
    assert torch.equal(i8.mx4_linear(torch.zeros((5, 0), dtype=torch.float16, device="cuda"), f, bias.half()), bias.half().expand(5, 6))
    g = torch.zeros((0, 6), dtype=torch.float16, device="cuda")
    w = torch.ones((6, 40), dtype=torch.float16, device="cuda")
    gx, gw = i8.mx4_linear_backward(g, torch.zeros((0, 40), dtype=torch.float16, device="cuda"), w)
    assert gx.shape == (0, 40) and gw.shape == (6, 40) and not gw.any()
    g = torch.zeros((7, 0), dtype=torch.float16, device="cuda")
    gx, gw = i8.mx4_linear_backward(g, torch.ones((7, 40), dtype=torch.float16, device="cuda"), w[:0])
    assert gx.shape == (7, 40) and not gx.any() and gw.shape == (0, 40)


# ---- products ---------------------------------------------------------------------

# rows of a, rows of b, k: single rows, edges of every tile, odd sizes, long sums
PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 100, 5120), (2, 257, 384), (3, 65, 129), (4, 1000, 1024), (8, 512, 13824), (15, 33, 640),
            (16, 1024, 2048), (17, 31, 255), (31, 200, 4096), (33, 63, 96), (48, 640, 896), (64, 128, 256), (65, 65, 257),
            (100, 300, 5000), (127, 129, 1023), (128, 4096, 512), (200, 1111, 777), (255, 513, 384), (256, 256, 1280),
            (257, 1025, 300), (512, 1536, 512), (1000, 96, 3333), (1025, 3000, 200), (2050, 4100, 130)]


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: "%dx%dx%d" % c)
def test_matmul_exact_sums(case):
    """Scales of 1, 2, 4: every sum is exact, whatever its order, so the result is the oracle's to the bit."""
    m, n, k = case
    rng = np.random.default_rng([83, *case])
    a, b = drawn(rng, m, k, 127, 130), drawn(rng, n, k, 126, 128)
    bias = rng.integers(-8, 9, n).astype(np.float32)
    want = mx4.values(*a)[:, :k] @ mx4.values(*b)[:, :k].T
    assert np.abs(want).max() < 2 ** 22
    say(f"mx4_matmul {case}")
    qa, qb = held(*a, k), held(*b, k)
    assert np.array_equal(wide(i8.mx4_matmul(qa, qb, dtype=torch.float32)), want)
    out = torch.full((m, n + 3), 5.0, device="cuda")
    i8.mx4_matmul(qa, qb, torch.from_numpy(bias).cuda(), torch.float32, out=out[:, 2:2 + n])
    assert np.array_equal(wide(out[:, 2:2 + n]), want + bias)
    assert bool((out[:, :2] == 5).all()) and bool((out[:, 2 + n:] == 5).all())
    for kind in ("f16", "bf16"):
        got = i8.mx4_matmul(qa, qb, torch.from_numpy(bias).cuda().to(DTYPE[kind]), DTYPE[kind])
        assert torch.equal(got.cpu(), torch.from_numpy((want + bias).astype(np.float32)).to(DTYPE[kind])), kind


# several tiles a workgroup, whole rounds and another cut for the last columns, sums split over k with every tile shape
LARGE = [(4352, 16640, 300), (4173, 22011, 1000), (8192, 2049, 1500), (1500, 1600, 5000), (40, 200, 20000), (100, 300, 9001),
         (512, 512, 60000), (128, 5120, 13824), (700, 1200, 9000), (300, 300, 30000), (17, 70001, 140), (70001, 17, 300)]


@pytest.mark.parametrize("case", LARGE, ids=lambda c: "%dx%dx%d" % c)
def test_matmul_exact_sums_large(case):
    """As above, against torch's fp32 product on the GPU, exact for such sums too."""
    m, n, k = case
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    kp = -(-k // 128) * 128
    lut = torch.tensor(np.concatenate([mx4.GRID, -mx4.GRID]), dtype=torch.float32, device="cuda")
    keep = torch.arange(kp, device="cuda") < k

    def drawn_here(rows, low, high):
        codes = torch.randint(0, 16, (rows, kp), generator=gen, device="cuda", dtype=torch.uint8) * keep
        # mostly small numbers where sums are long: they stay below 2^22 quarters
        if k > 5000:
            codes = torch.where(torch.rand(codes.shape, generator=gen, device="cuda") < 0.98, codes & 9, codes)
        scales = torch.randint(low, high, (rows, kp // 32), generator=gen, device="cuda", dtype=torch.uint8)
        value = lut[codes.int()] * torch.exp2(scales.float() - 127).repeat_interleave(32, 1)
        return i8.Mx4Tensor(codes[:, 0::2] | codes[:, 1::2] << 4, scales, k), value

    qa, a = drawn_here(m, 127, 129)
    qb, b = drawn_here(n, 126, 128)
    bias = torch.randint(-8, 9, (n,), generator=gen, device="cuda").float()
    say(f"mx4_matmul large {case}")
    want = a @ b.t()
    # what has passed through a sum on the way, in quarters of the least product, stays whole in fp32
    assert float((a.abs().max() * b.abs().max())) * k < 2 ** 24 or float((a.abs() @ b.abs().t()).max()) < 2 ** 22
    got = i8.mx4_matmul(qa, qb, dtype=torch.float32)
    assert torch.equal(got, want)
    out = torch.full((m, n + 5), 7.0, dtype=torch.float16, device="cuda")
    i8.mx4_matmul(qa, qb, bias.half(), out=out[:, 1:1 + n])
    assert torch.equal(out[:, 1:1 + n], (want + bias).half())
    assert bool((out[:, :1] == 7).all()) and bool((out[:, 1 + n:] == 7).all())
    assert torch.equal(i8.mx4_matmul(qa, qb, bias.bfloat16(), torch.bfloat16), (want + bias).bfloat16())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_outputs_larger_than_the_last_level_cache(kind):
    """Such results are stored another way; sums of whole quarters, exact in fp32."""
    m, n, k = 8500, 16904, 90
    gen = torch.Generator(device="cuda").manual_seed(96)
    grid = torch.tensor(np.concatenate([mx4.GRID, -mx4.GRID]), dtype=torch.float32, device="cuda")
    x, w = (grid[torch.randint(0, 16, (r, k), generator=gen, device="cuda")] for r in (m, n))
    for t in (x, w):
        t[:, ::32] = 6.0                                       # every block's scale is 1
    say(f"mx4_matmul past the cache {kind}")
    got = i8.mx4_matmul(i8.mx4_quantize(x.half()), i8.mx4_quantize(w.half()), dtype=DTYPE[kind])
    assert torch.equal(got, (x @ w.t()).to(DTYPE[kind]))


@pytest.mark.parametrize("m,n,k", [(1, 60, 600), (4, 90, 1152), (16, 40, 128), (40, 300, 600), (200, 260, 384), (800, 900, 640)])
def test_a_neighbours_scales_are_not_read_as_a_rows_own(m, n, k):
    """Rows that end in the middle of a stage of 256, beside rows that begin with a block that is no number."""
    rng = np.random.default_rng([93, m, k])
    a, b = drawn(rng, m, k), drawn(rng, n, k)
    a[1][1::2, 0] = 255
    b[1][2::3, 0] = 255
    say(f"mx4_matmul neighbours {m} {n} {k}")
    got = wide(i8.mx4_matmul(held(*a, k), held(*b, k), dtype=torch.float32))
    with np.errstate(invalid="ignore"):
        want = mx4.values(*a) @ mx4.values(*b).T
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


def test_large_outputs_of_dequantize():
    """Outputs past half the last-level cache are stored another way."""
    say("mx4_dequantize large")
    for m, k, t in ((6000, 11300, torch.float16), (6000, 5700, torch.float32), (5000, 13500, torch.bfloat16)):
        x = torch.randn((m, k), device="cuda", dtype=torch.float32).to(torch.float16)
        q = i8.mx4_quantize(x)
        got = i8.mx4_dequantize(q, t)
        rows = torch.tensor([0, 1, 777, m // 2, m - 1])
        assert np.array_equal(wide(got[rows.cuda()]), mx4.rounded(wide(x[rows.cuda()])))
        assert bool((got.float().abs().sum(1) > 0).all())


@pytest.mark.parametrize("case", [(1, 300, 5120), (5, 64, 1000), (40, 200, 4096), (130, 260, 2500), (300, 2000, 640)],
                         ids=lambda c: "%dx%dx%d" % c)
@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
def test_matmul_wide_scales(case, kind):
    m, n, k = case
    rng = np.random.default_rng([84, *case])
    a, b = drawn(rng, m, k, 110, 130), drawn(rng, n, k, 115, 127)
    say(f"mx4_matmul wide {case} {kind}")
    got = i8.mx4_matmul(held(*a, k, (16, 4)), held(*b, k, (48, 12)), dtype=DTYPE[kind])
    want, size = mx4.matmul(mx4.values(*a), mx4.values(*b))
    if kind == "f16":
        assert np.abs(want).max() < 65504
    close(got, want, size, a[0].shape[1], kind)


@pytest.mark.parametrize("m,n", [(1, 40), (20, 70), (150, 280), (600, 700)])
def test_blocks_that_are_no_numbers_stay_in_their_rows(m, n):
    rng = np.random.default_rng([85, m])
    k = 700
    a, b = drawn(rng, m, k), drawn(rng, n, k)
    a[1][m // 2, 3] = 255
    b[1][n - 1, 21] = 255
    b[1][n // 3, 0] = 255
    say(f"mx4_matmul nan {m} {n}")
    got = wide(i8.mx4_matmul(held(*a, k), held(*b, k), dtype=torch.float32))
    with np.errstate(invalid="ignore"):
        want = mx4.values(*a) @ mx4.values(*b).T
    assert np.isnan(want).sum() == n + 2 * m - 2
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


def test_range_of_the_sums():
    """fp32 sums: past 2^128 they are infinities, fp16 outputs overflow likewise; tiny ones stay."""
    say("mx4_matmul range")
    one = np.full((1, 128), 2, np.uint8)                       # ones
    def product(sa, sb, t):
        a = held(one, np.full((1, 4), sa), 128)
        b = held(one, np.full((1, 4), sb), 128)
        return wide(i8.mx4_matmul(a, b, dtype=t))[0, 0]
    assert product(254, 121, torch.float32) == np.inf and product(247, 120, torch.float32) == 2.0 ** 120
    assert product(127, 140, torch.float16) == np.inf and product(127, 135, torch.float16) == 2.0 ** 15
    assert product(1, 2, torch.float32) == 0.0 and product(60, 60, torch.float32) == 2.0 ** -127
    assert product(0, 127, torch.float32) == 2.0 ** -120


LINEARS = [(1, 64, 64), (1, 1000, 5120), (2, 333, 1111), (4, 512, 4096), (7, 130, 13824), (16, 640, 1000), (33, 257, 640),
           (128, 1024, 1024), (301, 555, 2000), (700, 1300, 333)]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("case", LINEARS, ids=lambda c: "%dx%dx%d" % c)
def test_linear(case, kind):
    m, n, k = case
    rng = np.random.default_rng([86, *case])
    x, w = rand16(rng, (m, k), kind, 1.0), rand16(rng, (n, k), kind) * 0.0625
    bias = rand16(rng, (n,), kind)
    wq = i8.mx4_quantize(dev16(w, kind))
    want, size = mx4.matmul(mx4.rounded(x), mx4.rounded(w))
    kp = -(-k // 128) * 128
    say(f"mx4_linear {case} {kind}")
    close(i8.mx4_linear(dev16(x, kind), wq), want, size, kp, kind)
    wider = dev16(np.pad(x, ((0, 0), (3, 2))), kind)[:, 3:3 + k]
    close(i8.mx4_linear(wider, wq, dev16(bias, kind)), want + bias, size + np.abs(bias), kp, kind)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 1), (1, 70, 200), (33, 64, 100), (130, 257, 300), (512, 384, 640), (1000, 200, 96)],
                         ids=lambda c: "%dx%dx%d" % c)
def test_linear_backward(case, kind):
    m, n, k = case
    rng = np.random.default_rng([87, *case])
    g, x, w = rand16(rng, (m, n), kind, 1.0), rand16(rng, (m, k), kind, 1.0), rand16(rng, (n, k), kind)
    say(f"mx4_linear_backward {case} {kind}")
    tg, tx, tw = dev16(g, kind), dev16(x, kind), dev16(w, kind)
    gx, gw = i8.mx4_linear_backward(tg, tx, tw)
    want, size = mx4.matmul(mx4.rounded(g), mx4.rounded(w.T))
    close(gx, want, size, -(-n // 128) * 128, kind)
    want, size = mx4.matmul(mx4.rounded(g.T), mx4.rounded(x.T))
    close(gw, want, size, -(-m // 128) * 128, kind)
    one, none = i8.mx4_linear_backward(tg, None, tw, need_grad_w=False)
    assert none is None and torch.equal(one, gx)
    none, one = i8.mx4_linear_backward(tg, tx, None, need_grad_x=False)
    assert none is None and torch.equal(one, gw)
    assert i8.mx4_linear_backward(tg, tx, tw, False, False) == (None, None)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("case", [(2560, 2816, 2816), (2047, 4100, 4090), (600, 4099, 1030), (4096, 300, 5000)],
                         ids=lambda c: "%dx%dx%d" % c)
def test_linear_backward_at_size(case, kind):
    """Both products in one launch, of large and of small tiles, into columns of wider matrices."""
    m, n, k = case
    gen = torch.Generator(device="cuda").manual_seed(m)
    g, x, w = (torch.randn(s, generator=gen, device="cuda").to(DTYPE[kind]) for s in ((m, n), (m, k), (n, k)))
    say(f"mx4_linear_backward at size {case} {kind}")
    bx, bw = (torch.full((r, k + 8), 7.0, dtype=DTYPE[kind], device="cuda") for r in (m, n))
    gx, gw = i8.mx4_linear_backward(g, x, w, out_x=bx[:, :k], out_w=bw[:, :k])
    assert gx.data_ptr() == bx.data_ptr() and gw.data_ptr() == bw.data_ptr()
    assert bool((bx[:, k:] == 7).all()) and bool((bw[:, k:] == 7).all())
    back = lambda t, columns: i8.mx4_dequantize(i8.mx4_quantize(t, columns), torch.float32).double()
    for got, a, b in ((gx, back(g, False), back(w, True)), (gw, back(g, True), back(x, True))):
        want, size = a @ b.t(), a.abs() @ b.abs().t()
        kp = -(-a.shape[1] // 128) * 128
        tol = (kp / 64 + 64) * 2.0 ** -23 * size + torch.finfo(DTYPE[kind]).eps / 2 * want.abs() + STEP[kind]
        assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,pitch", [(3000, 2701, 2701), (2500, 4096, 4100), (8000, 1100, 1128)])
def test_grad_out_by_rows_and_by_columns_at_once(m, n, pitch, kind):
    """A large grad_out is quantized both ways in one pass: every code shows in products with rows that are one block each."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    g = torch.randn((m, pitch), generator=gen, device="cuda").mul_(torch.exp2(torch.randint(-3, 4, (m, 1), generator=gen, device="cuda")))
    g = g.to(DTYPE[kind])[:, :n]
    g[5, 64:96], g[64:96, 7] = 0.0, 0.0
    g[m - 1, n - 1], g[9, 200] = float("nan"), float("inf")
    say(f"mx4_linear_backward both ways {m} {n} {kind}")
    x, w = (torch.randn((r, 24), generator=gen, device="cuda").to(DTYPE[kind]) for r in (m, n))
    gx, gw = i8.mx4_linear_backward(g, x, w)
    one = i8.mx4_linear_backward(g, None, w, need_grad_w=False)[0], i8.mx4_linear_backward(g, x, None, need_grad_x=False)[1]
    back = lambda t, columns: i8.mx4_dequantize(i8.mx4_quantize(t, columns), torch.float32).double()
    for got, a, b, same in ((gx, back(g, False), back(w, True), one[0]), (gw, back(g, True), back(x, True), one[1])):
        bad = a.isnan().any(1)
        assert int(bad.sum()) == 2 and bool(got[bad].isnan().all()) and bool(same[bad].isnan().all())
        want, size = a[~bad] @ b.t(), a[~bad].abs() @ b.abs().t()
        tol = (-(-a.shape[1] // 128) * 2 + 64) * 2.0 ** -23 * size + torch.finfo(DTYPE[kind]).eps / 2 * want.abs() + STEP[kind]
        for t in (got, same):
            assert bool(((t[~bad].double() - want).abs() <= tol).all())


def test_gradients_are_differences_of_the_linear():
    """Where every operand is on the 4-bit grid, the linear is linear and its gradients are its differences."""
    rng = np.random.default_rng(88)
    m, n, k = 40, 50, 70
    x, w, g = (rng.choice(np.concatenate([mx4.GRID, -mx4.GRID]), s) for s in ((m, k), (n, k), (m, n)))
    for t in (x, w, g):                                        # every block, along rows and columns, reaches 6 or 4: scale 1
        t[:, ::16] = 6.0
        t[::16, :] = 4.0
    dev = lambda a: dev16(a.astype(np.float32), "f16")
    say("mx4_linear_backward differences")
    gx, gw = (wide(t) for t in i8.mx4_linear_backward(dev(g), dev(x), dev(w)))

    def loss(xx, ww):                                          # sum of g out: out's rounding is none (whole quarters)
        q = i8.mx4_quantize(dev(xx)), i8.mx4_quantize(dev(ww))
        return float((wide(i8.mx4_matmul(*q, dtype=torch.float32)) * g).sum())

    base = loss(x, w)
    for i, j in ((1, 1), (3, 5), (39, 69), (17, 33)):
        for which in (0, 1):
            t = [x.copy(), w.copy()]
            old = t[which][i, j]
            t[which][i, j] = 4.0 if old == 6.0 else 6.0
            step = t[which][i, j] - old
            grad = ((gx, gw)[which][i, j], (g @ w, g.T @ x)[which][i, j])
            assert (loss(*t) - base) / step == grad[1]
            assert abs(grad[0] - grad[1]) <= 2.0 ** -11 * abs(grad[1])


def test_workspaces_streams_and_graphs():
    """A caller's workspace, another stream, and captured calls that are replayed between eager ones."""
    rng = np.random.default_rng(89)
    cases = [(1, 500, 2048), (3, 64, 8192), (40, 300, 4096), (300, 600, 1000)]
    lib = i8._lib.lib()
    stream = torch.cuda.Stream()
    for m, n, k in cases:
        xs = [dev16(rand16(rng, (m, k), "f16", 1.0), "f16") for _ in range(4)]
        w16 = dev16(rand16(rng, (n, k), "f16"), "f16")
        g = dev16(rand16(rng, (m, n), "f16"), "f16")
        w = i8.mx4_quantize(w16)
        say(f"mx4 graph {m} {n} {k}")
        want = [(i8.mx4_linear(x, w), *i8.mx4_linear_backward(g, x, w16)) for x in xs]
        ws = torch.full((max(lib.i8mp_mx4_linear_workspace_bytes(m, n, k), 1),), 255, dtype=torch.uint8, device="cuda")
        wb = torch.full((lib.i8mp_mx4_linear_backward_workspace_bytes(m, n, k),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        x, graph = xs[0].clone(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            assert torch.equal(i8.mx4_linear(x, w, workspace=ws), want[0][0])
            with torch.cuda.graph(graph, stream=stream):
                got = (i8.mx4_linear(x, w, workspace=ws), *i8.mx4_linear_backward(g, x, w16, workspace=wb))
        torch.cuda.synchronize()
        for x_new, expect in zip(xs, want):
            x.copy_(x_new)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, expect):
                assert torch.equal(a, b)
            assert torch.equal(i8.mx4_linear(x_new, w), expect[0])


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    w = i8.mx4_quantize(x)
    for f, error in ((lambda: i8.mx4_quantize(x.float()), TypeError), (lambda: i8.mx4_quantize(x.t()), ValueError),
                     (lambda: i8.mx4_quantize(x[:1].expand(4, 64)), ValueError),
                     (lambda: i8.mx4_quantize(x, out=i8.Mx4Tensor.create(4, 65)), ValueError),
                     (lambda: i8.mx4_dequantize(w, torch.int8), ValueError),
                     (lambda: i8.mx4_dequantize(w, out=torch.zeros((4, 63), dtype=torch.float16, device="cuda")), ValueError),
                     (lambda: i8.mx4_matmul(w, i8.Mx4Tensor.create(4, 65)), ValueError),
                     (lambda: i8.mx4_matmul(w, w, torch.zeros(4, device="cuda")), ValueError),
                     (lambda: i8.mx4_matmul(w, w, dtype=torch.float64), ValueError),
                     (lambda: i8.mx4_matmul(w, w, out=torch.zeros((4, 5), dtype=torch.float16, device="cuda")), ValueError),
                     (lambda: i8.mx4_linear(x.bfloat16(), w, torch.zeros(4, dtype=torch.float16, device="cuda")), ValueError),
                     (lambda: i8.mx4_linear(x[:, :60], w), ValueError),
                     (lambda: i8.mx4_linear(x, w, workspace=torch.zeros(8, device="cuda")), ValueError),
                     (lambda: i8.mx4_linear(x, i8.Mx4Tensor(w.codes[:, 1:], w.scales, 64)), ValueError),
                     (lambda: i8.mx4_linear_backward(x, x, x.bfloat16()), TypeError),
                     (lambda: i8.mx4_linear_backward(x, None, x), ValueError),
                     (lambda: i8.mx4_linear_backward(x, x[:3], x), ValueError),
                     (lambda: i8.mx4_matmul(w, i8.Mx4Tensor(w.codes.cpu(), w.scales, 64)), ValueError)):
        with pytest.raises(error):
            f()
