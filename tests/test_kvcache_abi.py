"""Host checks of the 4-bit key/value cache's entry points: every call below fails
validation (or, without a GPU, the device check) before anything is enqueued."""

import ctypes

import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from int8_mixed_precision_vectorwise_amd import _lib

OK, EINVAL, EWORKSPACE, EDEVICE = 0, -1, -3, -4
A16, ODD = 0x1000, 0x1008


def cache(**kw):
    f = dict(data=A16, pages=10, kv_heads=2, page_size=64, head_dim=128, dtype=0)
    f.update(kw)
    return _lib.Fp4CacheStruct(**f)


def call(**kw):
    f = dict(q=A16, ldq=512, hsq=128, out=A16, ldo=512, hso=128, lse=None, table=A16, ldt=8, table_cols=8, lengths=A16,
             q_offsets=None, alibi=None, prefix=None, tokens=3, batch=3, q_heads=4, max_q=1, max_len=512, window=0,
             scale=0.1, softcap=0.0)
    f.update(kw)
    return _lib.Fp4AttentionStruct(**f)


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def ref(x):
    return None if x is None else ctypes.byref(x)


BAD_CACHES = [dict(pages=0), dict(pages=1 << 31), dict(kv_heads=0), dict(kv_heads=65536), dict(page_size=8),
              dict(page_size=48), dict(page_size=512), dict(page_size=0), dict(head_dim=96), dict(head_dim=192),
              dict(head_dim=512), dict(dtype=1), dict(dtype=3)]


def test_cache_bytes(L):
    for page in (16, 32, 64, 128, 256):
        for d in (64, 128, 256):
            for dtype in (0, 2):
                assert L.i8mp_fp4_cache_bytes(ref(cache(page_size=page, head_dim=d, dtype=dtype, data=None))) == \
                    10 * 2 * page * 68 * d // 64
    assert L.i8mp_fp4_cache_bytes(ref(cache(pages=1 << 30))) == (1 << 30) * 2 * 64 * 136
    for bad in BAD_CACHES:
        assert L.i8mp_fp4_cache_bytes(ref(cache(**bad))) == 0, bad
    assert L.i8mp_fp4_cache_bytes(None) == 0


def test_move_validation(L):
    w, r = L.i8mp_fp4_cache_write, L.i8mp_fp4_cache_read
    good = (A16, 256, 128, A16, 256, 128, A16, 4, None)
    for bad in BAD_CACHES:
        assert w(ref(cache(**bad)), *good) == EINVAL, bad
        assert r(ref(cache(**bad)), A16, 4, 0, A16, 256, 128, A16, 256, 128, None) == EINVAL, bad
    assert w(None, *good) == EINVAL
    for i, x in ((0, None), (3, None), (6, None), (0, ODD), (3, ODD), (1, 120), (1, 260), (2, 127), (2, 132), (4, 100),
                 (5, 64), (7, -1)):
        args = list(good)
        args[i] = x
        assert w(ref(cache()), *args) == EINVAL, (i, x)
    assert w(ref(cache(data=None)), *good) == EINVAL and w(ref(cache(data=ODD)), *good) == EINVAL
    assert w(ref(cache()), None, 256, 128, None, 256, 128, None, 0, None) == OK
    good = (A16, 4, 1, A16, 256, 128, A16, 256, 128, None)
    for i, x in ((0, None), (1, -1), (2, 3), (2, -1), (3, None), (3, ODD), (4, 127), (4, 258), (5, 130), (6, None),
                 (7, 1), (8, 0)):
        args = list(good)
        args[i] = x
        assert r(ref(cache()), *args) == EINVAL, (i, x)
    assert r(ref(cache()), A16, 4, 0, A16, 260, 128, A16, 256, 128, None) == EINVAL     # a multiple of 4 only for fp32
    assert r(ref(cache()), None, 0, 2, None, 256, 128, None, 256, 128, None) == OK
    if torch.cuda.device_count() == 0:
        assert r(ref(cache()), A16, 4, 1, A16, 260, 132, A16, 256, 128, None) == EDEVICE
        assert w(ref(cache()), A16, 256, 128, A16, 256, 128, A16, 4, None) == EDEVICE


def test_attention_validation(L):
    run, need = L.i8mp_fp4_cache_attention, L.i8mp_fp4_attention_workspace_bytes

    def status(c=None, ws=A16, wsb=1 << 40, **kw):
        return run(ref(c or cache()), ref(call(**kw)), ws, wsb, None)

    for bad in BAD_CACHES:
        assert status(cache(**bad)) == EINVAL and need(ref(cache(**bad)), ref(call())) == 0, bad
    assert run(None, ref(call()), A16, 1 << 40, None) == EINVAL and run(ref(cache()), None, A16, 1 << 40, None) == EINVAL
    for bad in (dict(q=None), dict(out=None), dict(table=None), dict(lengths=None), dict(q=ODD), dict(out=ODD),
                dict(ldq=127), dict(ldq=516), dict(hsq=64), dict(hsq=130), dict(ldo=511), dict(hso=127), dict(tokens=-1),
                dict(tokens=4), dict(batch=-1), dict(q_heads=3), dict(q_heads=0), dict(q_heads=1 << 17), dict(max_q=0),
                dict(max_len=513), dict(max_len=-1), dict(window=-1), dict(table_cols=-1), dict(ldt=7),
                dict(scale=float("nan")), dict(softcap=-1.0), dict(softcap=float("inf")),
                dict(max_len=(1 << 30) + 1, table_cols=1 << 30, ldt=1 << 30),
                dict(q_offsets=A16, max_q=1 << 30), dict(q_offsets=A16, max_q=1 << 29, batch=32, tokens=32)):
        assert status(**bad) == EINVAL, bad
    assert status(batch=0, tokens=0, q=None, out=None) == OK
    assert status(batch=2, tokens=0, q_offsets=A16, q=None, out=None) == OK
    long = dict(batch=1, tokens=1, table_cols=1 << 14, ldt=1 << 14, max_len=1 << 20)
    n = need(ref(cache()), ref(call(**long)))
    assert n > 0 and need(ref(cache()), ref(call(batch=0, tokens=0))) == 0
    assert status(ws=None, wsb=0, **long) == EWORKSPACE and status(wsb=n - 1, **long) == EWORKSPACE
    assert status(ws=ODD, wsb=n, **long) == EWORKSPACE
    if torch.cuda.device_count() == 0:
        assert status(wsb=n, **long) == EDEVICE and status() == EDEVICE


def test_python_binding_refuses_cpu_tensors_and_bad_caches():
    c = i8.Fp4Cache.create(2, 1, 64, 16, device="cpu")
    x = torch.zeros((1, 1, 64), dtype=torch.float16)
    slots = torch.zeros(1, dtype=torch.int64)
    i32 = torch.zeros(1, dtype=torch.int32)
    for f in (lambda: i8.fp4_cache_write(c, x, x, slots), lambda: i8.fp4_cache_read(c, slots),
              lambda: i8.fp4_cache_attention(x, c, i32.view(1, 1), i32)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    for bad in (dict(head_dim=96), dict(page_size=24), dict(page_size=512), dict(head_dim=512)):
        with pytest.raises(ValueError):
            i8.Fp4Cache.create(**{**dict(pages=2, kv_heads=1, head_dim=64, page_size=16, device="cpu"), **bad})
    with pytest.raises(TypeError):
        i8.Fp4Cache.create(2, 1, 64, 16, torch.float32, device="cpu")
    with pytest.raises(ValueError):
        i8.Fp4Cache(c.data[:, :, :-1], 16, 64).struct()
    with pytest.raises(ValueError):
        i8.Fp4Cache(c.data, 32, 64).struct()
