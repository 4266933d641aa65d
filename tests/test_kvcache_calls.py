"""Host side of the 4-bit cache's calls: what they ask for and what they refuse."""

import pytest

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
