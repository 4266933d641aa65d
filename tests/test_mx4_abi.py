"""Host checks of the microscaled matrices' entry points and of the append to the 4-bit
cache: every call below fails validation (or, without a GPU, the device check) before
anything is enqueued."""

import ctypes

import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from int8_mixed_precision_vectorwise_amd import _lib
from test_kvcache_abi import BAD_CACHES, cache

OK, EINVAL, EWORKSPACE, EDEVICE = 0, -1, -3, -4
A16, ODD, BYTE = 0x1000, 0x1008, 0x1001
NO_GPU = torch.cuda.device_count() == 0
BIG = 1 << 40


def mx(**kw):
    f = dict(codes=A16, scales=A16, rows=5, k=200, ldc=128, lds=8)
    f.update(kw)
    return ctypes.byref(_lib.Mx4Struct(**f))


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


BAD = [dict(rows=-1), dict(rows=1 << 31), dict(k=-1), dict(ldc=127), dict(ldc=112), dict(ldc=136), dict(lds=4),
       dict(lds=10), dict(ldc=(1 << 20) + 16), dict(lds=(1 << 20) + 4), dict(k=257)]
BAD_DATA = [dict(codes=None), dict(scales=None), dict(codes=ODD), dict(scales=BYTE)]


def test_quantize_and_dequantize_validation(L):
    quant, back = L.i8mp_mx4_quantize, L.i8mp_mx4_dequantize
    for bad in BAD + BAD_DATA:
        assert quant(A16, 0, 5, 200, 200, 0, mx(**bad), None) == EINVAL, bad
        assert back(mx(**bad), 0, A16, 257, None) == EINVAL, bad
    assert quant(A16, 0, 5, 200, 200, 0, None, None) == EINVAL and back(None, 0, A16, 200, None) == EINVAL
    good = [A16, 0, 5, 200, 200, 0]
    for i, x in ((0, None), (1, 1), (1, 3), (2, 4), (2, -1), (3, 199), (4, 199), (5, 1)):
        args = list(good)
        args[i] = x
        assert quant(*args, mx(), None) == EINVAL, (i, x)
    assert quant(A16, 0, 200, 5, 5, 0, mx(), None) == EINVAL            # a transpose that is not asked for
    for x in (-1, 3):
        assert back(mx(), x, A16, 200, None) == EINVAL
    assert back(mx(), 0, A16, 199, None) == EINVAL and back(mx(), 0, None, 200, None) == EINVAL
    assert quant(None, 0, 0, 200, 200, 0, mx(rows=0, codes=None, scales=None), None) == OK
    assert quant(None, 2, 5, 0, 0, 0, mx(k=0, ldc=0, lds=0, codes=None, scales=None), None) == OK
    assert back(mx(rows=0), 1, None, 200, None) == OK
    if NO_GPU:
        assert quant(BYTE + 1, 2, 200, 5, 5, 1, mx(), None) == EDEVICE
        assert quant(A16, 0, 5, 200, 999, 0, mx(ldc=1 << 20, lds=1 << 20), None) == EDEVICE
        assert back(mx(), 1, A16, 200, None) == EDEVICE


def test_matmul_validation(L):
    run, need = L.i8mp_mx4_matmul, L.i8mp_mx4_matmul_workspace_bytes

    def status(a=None, b=None, bias=None, dtype=0, out=A16, ldout=7, ws=A16, wsb=BIG):
        return run(a or mx(), b or mx(rows=7), bias, dtype, out, ldout, ws, wsb, None)

    for bad in BAD + BAD_DATA:
        assert status(a=mx(**bad)) == EINVAL and status(b=mx(**{**dict(rows=7), **bad})) == EINVAL, bad
    assert run(None, mx(), None, 0, A16, 7, A16, BIG, None) == EINVAL and run(mx(), None, None, 0, A16, 7, A16, BIG, None) == EINVAL
    assert status(b=mx(rows=7, k=199)) == EINVAL
    for bad in (dict(dtype=3), dict(dtype=-1), dict(out=None), dict(ldout=6), dict(ldout=(1 << 20) + 1)):
        assert status(**bad) == EINVAL, bad
    assert status(a=mx(rows=0, codes=None), out=None) == OK and status(b=mx(rows=0, scales=None), out=None) == OK
    for m, n, k in ((-1, 5, 5), (5, -1, 5), (5, 5, -1), (1 << 31, 5, 5), (5, 1 << 31, 5), (5, 5, 1 << 31)):
        assert need(m, n, k) == 0
        assert L.i8mp_mx4_linear_workspace_bytes(m, n, k) == 0 and L.i8mp_mx4_linear_backward_workspace_bytes(m, n, k) == 0
    if NO_GPU:
        assert status() == EDEVICE and status(a=mx(k=0), b=mx(k=0, rows=7), bias=A16, dtype=1) == EDEVICE


def test_matmul_workspace(L):
    """Where sums are split over k, the parts take space: NULL, too little and a misaligned one are refused."""
    run, need = L.i8mp_mx4_matmul, L.i8mp_mx4_matmul_workspace_bytes
    seen = 0
    for m, n, k in ((5, 7, 200), (1, 64, 131072), (64, 64, 131072), (300, 200, 65536), (4096, 22016, 8192)):
        w = need(m, n, k)
        kp = -(-k // 128) * 128
        a, b = mx(rows=m, k=k, ldc=kp // 2, lds=kp // 32), mx(rows=n, k=k, ldc=kp // 2, lds=kp // 32)
        if w:
            seen += 1
            assert run(a, b, None, 0, A16, n, None, 0, None) == EWORKSPACE
            assert run(a, b, None, 0, A16, n, A16, w - 1, None) == EWORKSPACE
            assert run(a, b, None, 0, A16, n, ODD, w, None) == EWORKSPACE
        if NO_GPU:
            assert run(a, b, None, 0, A16, n, A16, w, None) == EDEVICE
    assert seen >= 2


def test_linear_validation(L):
    run, need = L.i8mp_mx4_linear, L.i8mp_mx4_linear_workspace_bytes

    def status(x=A16, dtype=0, m=5, ldx=200, w=None, bias=None, out=A16, ldout=7, ws=A16, wsb=BIG):
        return run(x, dtype, m, ldx, w or mx(rows=7), bias, out, ldout, ws, wsb, None)

    for bad in BAD + BAD_DATA:
        assert status(w=mx(**{**dict(rows=7), **bad})) == EINVAL, bad
    for bad in (dict(x=None), dict(dtype=1), dict(dtype=4), dict(m=-1), dict(m=1 << 31), dict(ldx=199), dict(out=None),
                dict(ldout=6), dict(ldout=(1 << 20) + 1)):
        assert status(**bad) == EINVAL, bad
    assert run(A16, 0, 5, 200, None, None, A16, 7, A16, BIG, None) == EINVAL
    assert status(m=0, x=None, out=None) == OK and status(w=mx(rows=0), out=None) == OK
    w = need(500, 700, 200)
    assert w >= 500 * (128 + 8)
    kw = dict(m=500, w=mx(rows=700), ldout=700)
    assert status(ws=None, wsb=0, **kw) == EWORKSPACE and status(wsb=w - 1, **kw) == EWORKSPACE
    assert status(ws=ODD, wsb=w, **kw) == EWORKSPACE
    if NO_GPU:
        assert status(wsb=w, **kw) == EDEVICE and status() == EDEVICE


def test_backward_validation(L):
    run, need = L.i8mp_mx4_linear_backward, L.i8mp_mx4_linear_backward_workspace_bytes

    def status(g=A16, ldg=7, x=A16, ldx=9, w=A16, ldw=9, dtype=0, m=5, n=7, k=9, gx=A16, ldgx=9, gw=A16, ldgw=9, ws=A16, wsb=BIG):
        return run(g, ldg, x, ldx, w, ldw, dtype, m, n, k, gx, ldgx, gw, ldgw, ws, wsb, None)

    for bad in (dict(g=None), dict(ldg=6), dict(x=None), dict(ldx=8), dict(w=None), dict(ldw=8), dict(dtype=1), dict(dtype=-1),
                dict(m=-1), dict(n=-1), dict(k=-1), dict(m=(1 << 21) + 1), dict(n=(1 << 21) + 1, ldg=1 << 22), dict(k=1 << 31),
                dict(ldgx=8), dict(ldgw=8), dict(ldgx=(1 << 20) + 1), dict(ldgw=(1 << 20) + 1)):
        assert status(**bad) == EINVAL, bad
    assert status(gx=None, gw=None, ws=None, wsb=0) == OK
    assert status(k=0, g=None, x=None, w=None, ws=None, wsb=0) == OK
    assert status(m=0, gw=None, ws=None, wsb=0) == OK and status(n=0, gx=None, ws=None, wsb=0) == OK
    n = need(5, 7, 9)
    assert status(wsb=n - 1) == EWORKSPACE and status(ws=None, wsb=0) == EWORKSPACE and status(ws=ODD, wsb=n) == EWORKSPACE
    if NO_GPU:
        assert status(wsb=n) == EDEVICE
        assert status(x=None, ldx=0, gw=None, ldgw=0) == EDEVICE and status(w=None, ldw=0, gx=None, ldgx=0) == EDEVICE


def test_append_validation(L):
    def status(c=None, **kw):
        f = dict(k=A16, ldk=256, hsk=128, v=A16, ldv=256, hsv=128, slots=A16, positions=A16, cos=A16, sin=A16, ldcos=64, ldsin=64,
                 table_rows=9, q=A16, ldq=512, hsq=128, out=A16, ldo=512, hso=128, tokens=4, q_heads=4, rotary=128, interleaved=0)
        f.update(kw)
        return L.i8mp_fp4_cache_append(ctypes.byref(c or cache()), ctypes.byref(_lib.Fp4AppendStruct(**f)), None)

    for bad in BAD_CACHES + [dict(data=None), dict(data=ODD)]:
        assert status(cache(**bad)) == EINVAL, bad
    for bad in (dict(k=None), dict(k=ODD), dict(v=None), dict(v=ODD), dict(slots=None), dict(positions=None), dict(cos=None),
                dict(sin=None), dict(ldk=120), dict(hsk=130), dict(ldv=127), dict(hsv=64), dict(ldcos=63), dict(ldsin=63),
                dict(table_rows=0), dict(q=None), dict(q=ODD), dict(out=None), dict(out=ODD), dict(ldq=100), dict(hsq=132),
                dict(ldo=127), dict(hso=4), dict(tokens=-1), dict(q_heads=-1), dict(q_heads=65536), dict(rotary=0),
                dict(rotary=8), dict(rotary=24), dict(rotary=144), dict(rotary=-16)):
        assert status(**bad) == EINVAL, bad
    assert L.i8mp_fp4_cache_append(None, None, None) == EINVAL
    assert L.i8mp_fp4_cache_append(ctypes.byref(cache()), None, None) == EINVAL
    assert status(tokens=0, k=None, v=None, slots=None, q=None, out=None) == OK
    if NO_GPU:
        assert status() == EDEVICE and status(q_heads=0, q=None, out=None, ldq=0, rotary=16, interleaved=1) == EDEVICE


def test_python_binding_refusals():
    x = torch.zeros((4, 64), dtype=torch.float16)
    w = i8.Mx4Tensor.create(4, 64, device="cpu")
    for f in (lambda: i8.mx4_quantize(x), lambda: i8.mx4_dequantize(w), lambda: i8.mx4_matmul(w, w), lambda: i8.mx4_linear(x, w),
              lambda: i8.mx4_linear_backward(x, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    c = i8.Fp4Cache.create(2, 1, 64, 16, device="cpu")
    h, i, t = torch.zeros((1, 1, 64), dtype=torch.float16), torch.zeros(1, dtype=torch.int64), torch.zeros((1, 32))
    with pytest.raises(ValueError, match="GPU"):
        i8.fp4_cache_append(c, h, h, h, i, i, t, t)
    assert w.shape == (4, 64) and w.rows == 4 and w.codes.shape == (4, 64) and w.scales.shape == (4, 4)
    for bad in (i8.Mx4Tensor(w.codes, w.scales, 129), i8.Mx4Tensor(w.codes, w.scales[:3], 64),
                i8.Mx4Tensor(w.codes, w.scales[:1].expand(4, 4), 64), i8.Mx4Tensor(w.codes[:, ::2], w.scales, 64)):
        with pytest.raises(ValueError):
            bad.struct()
    with pytest.raises(TypeError):
        i8.Mx4Tensor(w.codes.to(torch.int8), w.scales, 64).struct()


def test_rows_that_a_grid_cannot_hold(L):
    most = 1 << 26
    assert L.i8mp_mx4_quantize(A16, 0, most + 1, 200, 200, 0, mx(rows=most + 1), None) == EINVAL
    assert L.i8mp_mx4_matmul(mx(rows=most + 1), mx(), None, 0, A16, 5, A16, BIG, None) == EINVAL
    assert L.i8mp_mx4_linear(A16, 0, most + 1, 200, mx(), None, A16, 5, A16, BIG, None) == EINVAL
    assert L.i8mp_mx4_linear_workspace_bytes(most + 1, 5, 200) == 0 < L.i8mp_mx4_linear_workspace_bytes(most, 5, 200)
    if NO_GPU:
        assert L.i8mp_mx4_quantize(A16, 0, most, 200, 200, 0, mx(rows=most), None) == EDEVICE
        assert L.i8mp_mx4_matmul(mx(rows=most), mx(), None, 0, A16, 5, A16, BIG, None) == EDEVICE


def test_few_rows_need_no_workspace(L):
    for k in (1, 200, 5120, 13824):
        assert L.i8mp_mx4_linear_workspace_bytes(4, 7, k) == 0 < L.i8mp_mx4_linear_workspace_bytes(5, 7, k)
    assert L.i8mp_mx4_linear_workspace_bytes(1, 7, 1 << 21) > 0          # more than LDS holds
    if NO_GPU:
        assert L.i8mp_mx4_linear(A16 + 2, 0, 4, 203, mx(rows=7), None, A16, 7, None, 0, None) == EDEVICE


def test_rows_whose_padded_length_leaves_64_bits(L):
    """k + 127 past 2^63 would be a small padded length, which any matrix holds."""
    top = (1 << 63) - 1
    for k in (top, top - 126, top - 127, (1 << 21) + 1):
        a, wide = mx(k=k), dict(ldc=1 << 20, lds=1 << 20)
        for m in (a, mx(k=k, **wide)):
            assert L.i8mp_mx4_quantize(A16, 0, 5, k, k, 0, m, None) == EINVAL, k
            assert L.i8mp_mx4_quantize(A16, 0, k, 5, 5, 1, m, None) == EINVAL, k
            assert L.i8mp_mx4_dequantize(m, 0, A16, k, None) == EINVAL, k
            assert L.i8mp_mx4_matmul(m, m, None, 0, A16, 5, A16, BIG, None) == EINVAL, k
            assert L.i8mp_mx4_linear(A16, 0, 5, k, m, None, A16, 5, A16, BIG, None) == EINVAL, k
    if NO_GPU:
        assert L.i8mp_mx4_quantize(A16, 0, 5, 1 << 21, 1 << 21, 0, mx(k=1 << 21, **wide), None) == EDEVICE


def test_tables_wider_than_the_c_call_can_say(monkeypatch):
    """ctypes keeps an int's low 32 bits: tables of 2^31 + 64 columns would turn 128 dims."""
    def refuse(*a):
        raise AssertionError("the call must not reach the library")

    monkeypatch.setattr(i8, "_device_of", lambda *t: torch.device("cuda", 0))
    monkeypatch.setattr(i8, "_run", refuse)
    c = i8.Fp4Cache.create(2, 1, 128, 16, device="cpu")
    h, i = torch.zeros((1, 1, 128), dtype=torch.float16), torch.zeros(1, dtype=torch.int64)
    for half in ((1 << 31) + 64, 1 << 30):
        t = torch.empty((1, half), device="meta")
        with pytest.raises(ValueError, match="rotary is out of range"):
            i8.fp4_cache_append(c, h, h, h, i, i, t, t)
