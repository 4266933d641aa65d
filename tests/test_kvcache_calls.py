"""Host side of the 4-bit cache's calls: what they ask for and what they refuse."""

import os
import subprocess
import sys

import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from int8_mixed_precision_vectorwise_amd import _lib
from test_kvcache_abi import A16, cache, call, ref


@pytest.mark.parametrize("d,kv_heads,group,batch,max_q", [
    (128, 8, 8, 64, 1), (128, 8, 8, 16, 1), (128, 8, 4, 4, 128), (128, 8, 8, 8, 12), (64, 8, 8, 1, 1), (256, 4, 4, 8, 4)])
def test_workspace_of_a_window_and_a_prefix_does_not_grow_with_the_table(d, kv_heads, group, batch, max_q):
    """What a row can see is the window and a prefix that only the device knows: tokens beside them take no space."""
    need = _lib.lib().i8mp_fp4_attention_workspace_bytes
    sizes = []
    for cols in (1 << 11, 1 << 12, 1 << 14, 1 << 18):
        c = cache(pages=1 << 20, kv_heads=kv_heads, head_dim=d)
        p = call(ldq=kv_heads * group * d, hsq=d, ldo=kv_heads * group * d, hso=d, tokens=batch * max_q, batch=batch,
                 max_q=max_q, q_heads=kv_heads * group, table_cols=cols, ldt=cols, max_len=cols * 64, window=1024, prefix=A16)
        sizes.append(need(ref(c), ref(p)))
    assert len(set(sizes)) == 1, sizes
    assert sizes[0] <= 64 << 20


def test_rows_that_overlap_are_refused():
    """An expanded table has one row in memory: as rows of its width it would be read past its end."""
    one = torch.zeros((1, 5), dtype=torch.int32)
    for t in (one.expand(3, 5), torch.zeros(9, dtype=torch.int32).as_strided((3, 5), (2, 1)), torch.zeros((1, 1), dtype=torch.int32).expand(4, 1)):
        with pytest.raises(ValueError, match="overlap"):
            i8._rowmajor(t, "table", torch.int32)
    assert i8._rowmajor(one, "table", torch.int32) == 5
    assert i8._rowmajor(one.expand(1, 5), "table", torch.int32) == 5
    assert i8._rowmajor(torch.zeros((4, 9), dtype=torch.int32)[:, :5], "table", torch.int32) == 9
    assert i8._rowmajor(torch.zeros((0, 5), dtype=torch.int32), "table", torch.int32) == 5
    assert i8._rowmajor(torch.zeros((3, 0), dtype=torch.int32), "table", torch.int32) == 1
    assert i8._rowmajor(torch.zeros((3, 1), dtype=torch.int32), "table", torch.int32) == 1


def test_a_workspace_is_a_run_of_bytes():
    """numel() is taken for the bytes that may be written: not so for an expanded tensor, or one with gaps."""
    for t in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(64, dtype=torch.uint8)[::2],
              torch.zeros(64), torch.zeros((8, 8), dtype=torch.uint8).t()):
        with pytest.raises(ValueError, match="workspace must be a contiguous"):
            i8._bytes(t, "workspace")
    i8._bytes(torch.zeros((4, 16), dtype=torch.uint8)[1:], "workspace")


def test_values_that_the_c_call_cannot_hold():
    """ctypes keeps an int's low 32 bits (a window of 2^32 + 1 became one of 1) and rounds a tiny cap to none."""
    call_ = _lib.Fp4AttentionStruct(window=(1 << 32) + 1, softcap=1e-50)
    assert call_.window == 1 and call_.softcap == 0.0
    for bad in ((1 << 32) + 1, 1 << 31, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="window is out of range"):
            i8._int32(max_q=1, window=bad)
    i8._int32(a=(1 << 31) - 1, b=-(1 << 31), c=0)
    for bad in (1e-50, -1e-50):
        with pytest.raises(ValueError, match="softcap is less"):
            i8._float32(softcap=bad)
    i8._float32(a=0.0, b=1e-44, c=float("nan"), d=1e60)


def test_the_package_imports_without_gpu_support_in_torch():
    """A torch built for the CPU alone has no raw stream handle."""
    code = ("import torch\n"
            "del torch._C._cuda_getCurrentRawStream\n"
            "import int8_mixed_precision_vectorwise_amd as i8\n"
            "c = i8.Fp4Cache.create(2, 1, 64, 16, device='cpu')\n"
            "try:\n    i8.fp4_cache_read(c, torch.zeros(1, dtype=torch.int64))\n"
            "except ValueError as e:\n    print('refused:', e)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "no CPU path" in r.stdout, r.stderr
