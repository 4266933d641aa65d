"""The attention block of the examples: prompts and single tokens through the int8
projections and the 4-bit cache, against the CPU oracle of the attention, to the
bounds of test_gpu_kvcache.py."""

import os
import sys

import numpy as np
import pytest
import torch

from gpu_util import host, say
from oracle import kvcache as kv
from test_gpu_kvcache import wide

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def bound(q, k, v, scale, window):
    """(oracle output, its bound) of queries whose last is the newest token: see test_gpu_kvcache.check."""
    o, _, size, reach = kv.attention(q, k, v, scale, window, 0.0, None, 0, None)
    e = 2.0 ** -24 * 260 * reach + 2.0 ** -20
    return o, 2.0 ** -11 * np.abs(o) + (2.0 ** -11 + 2 * e[..., None]) * size + 2.0 ** -23


@pytest.mark.parametrize("kv_heads,window", [(4, 0), (2, 25)])
def test_prompts_then_tokens(kv_heads, window):
    from attention_block import AttentionBlock

    hidden, heads, d, batch = 256, 4, 64, 3
    gen = torch.Generator(device="cuda").manual_seed(71)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    w_qkv = (rand((heads + 2 * kv_heads) * d, hidden) * hidden ** -0.5).half()
    w_out = (rand(hidden, heads * d) * hidden ** -0.5).half()
    block = AttentionBlock(w_qkv, w_out, heads, kv_heads, batch, 80, page_size=16, window=window)
    keep = []
    attend = block.attend

    def record(x, slots, q_offsets, max_q):       # q, k and v as the block's own projection gives them
        import int8_mixed_precision_vectorwise_amd as i8
        y = i8.linear(x, *block.qkv).view(x.shape[0], -1, d)
        out = attend(x, slots, q_offsets, max_q)
        keep.append(([wide(t) for t in y.split([heads, kv_heads, kv_heads], 1)], wide(out[1])))
        return out

    block.attend = record
    calls = [[40, 17, 0], [5, 0, 33], [1, 1, 1], [1, 1, 1], [9, 1, 2]]
    say(f"attention block, {heads} / {kv_heads} heads, window {window}")
    for n in calls:
        x = rand(sum(n), hidden).half()
        y, _ = block.step(x) if n == [1, 1, 1] else block.prompt(x, n)
        assert y.shape == (sum(n), hidden) and bool(torch.isfinite(y).all())
    torch.cuda.synchronize()
    assert host(block.lengths).tolist() == [56, 20, 37]
    ks, vs = [[] for _ in range(batch)], [[] for _ in range(batch)]
    for n, ((q, k, v), got) in zip(calls, keep):
        at = 0
        for b in range(batch):
            rows = slice(at, at + n[b])
            at += n[b]
            ks[b].append(kv.dequantize(*kv.quantize(k[rows])))
            vs[b].append(kv.dequantize(*kv.quantize(v[rows])))
            if n[b]:
                want, tol = bound(q[rows], np.concatenate(ks[b]), np.concatenate(vs[b]), d ** -0.5, window)
                assert np.all(np.abs(got[rows] - want) <= tol), (n, b)


def test_the_example_runs(capsys):
    from attention_block import main

    say("attention block: the command")
    main(["--hidden", "512", "--head-dim", "64", "--kv-heads", "2", "--batch", "3", "--prompt", "90", "--steps", "4"])
    assert "decode step" in capsys.readouterr().out
