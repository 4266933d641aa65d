"""The attention block of the examples with microscaled 4-bit projections and positions: prompts, then single tokens.

Each operator against its oracle, on what the one before it gave: the projections to the bound of test_gpu_mx4.py, the
attention over keys turned in 64 bits and quantized by the oracle to that of test_gpu_attention_block.py."""

import os
import sys

import numpy as np
import pytest
import torch

import int8_mixed_precision_vectorwise_amd as i8
from gpu_util import host, say
from oracle import kvcache as kv
from oracle import mx4
from test_gpu_attention_block import bound
from test_gpu_mx4 import close, wide

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

HIDDEN, HEADS, D, BATCH = 256, 4, 64, 3


def make(gen, kv_heads, rotary, window=0):
    from attention_block import AttentionBlock

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    w_qkv = (rand((HEADS + 2 * kv_heads) * D, HIDDEN) * HIDDEN ** -0.5).half()
    w_out = (rand(HIDDEN, HEADS * D) * HIDDEN ** -0.5).half()
    return AttentionBlock(w_qkv, w_out, HEADS, kv_heads, BATCH, 80, page_size=16, window=window, bits=4,
                          rotary=rotary), w_qkv, w_out, rand


@pytest.mark.parametrize("kv_heads,rotary,window", [(4, 64, 0), (2, 32, 25), (1, 0, 0)])
def test_prompts_then_tokens(kv_heads, rotary, window):
    block, w_qkv, w_out, rand = make(torch.Generator(device="cuda").manual_seed(94), kv_heads, rotary, window)
    wq, wo = mx4.rounded(wide(w_qkv)), mx4.rounded(wide(w_out))
    ks, vs = [[] for _ in range(BATCH)], [[] for _ in range(BATCH)]
    lengths = np.zeros(BATCH, int)
    say(f"4-bit attention block, {HEADS} / {kv_heads} heads, {rotary} dims turn, window {window}")
    for n in [[40, 17, 0], [5, 0, 33], [1, 1, 1], [1, 1, 1], [9, 1, 2]]:
        x = rand(sum(n), HIDDEN).half()
        y, a = block.step(x) if n == [1, 1, 1] else block.prompt(x, n)
        a = a.reshape(sum(n), -1)
        close(y, *mx4.matmul(mx4.rounded(wide(a)), wo), HEADS * D, "f16")
        got = i8.mx4_linear(x, *block.qkv)
        close(got, *mx4.matmul(mx4.rounded(wide(x)), wq), HIDDEN, "f16")
        q, k, v = np.split(wide(got).reshape(sum(n), -1, D), [HEADS, HEADS + kv_heads], 1)
        place = np.concatenate([lengths[b] + np.arange(n[b]) for b in range(BATCH)])
        if rotary:
            cos, sin = (host(t)[place] for t in (block.cos, block.sin))
            q, k = (kv.round16(mx4.rotate(t, cos, sin, False).astype(np.float32), "f16") for t in (q, k))
        at = 0
        for b in range(BATCH):
            rows = slice(at, at + n[b])
            at += n[b]
            ks[b].append(kv.dequantize(*kv.quantize(k[rows])))
            vs[b].append(kv.dequantize(*kv.quantize(v[rows])))
            if n[b]:
                want, tol = bound(q[rows], np.concatenate(ks[b]), np.concatenate(vs[b]), D ** -0.5, window)
                assert np.all(np.abs(wide(a)[rows].reshape(want.shape) - want) <= tol), (n, b)
        lengths += n
    assert host(block.lengths).tolist() == lengths.tolist()


def test_a_captured_step():
    """A step that projects, turns, writes, attends and projects, replayed with the program's own work between."""
    block, _, _, rand = make(torch.Generator(device="cuda").manual_seed(95), 2, 64)
    say("4-bit attention block: a captured step")
    block.prompt(rand(60, HIDDEN).half(), [30, 1, 29])
    xs = [rand(BATCH, HIDDEN).half() for _ in range(4)]
    start = block.lengths.clone(), block.cache.data.clone()

    def again():
        block.lengths.copy_(start[0])
        block.cache.data.copy_(start[1])

    want = []
    for x in xs:
        y, a = block.step(x)
        want.append((y.clone(), a.clone()))
    cache = block.cache.data.clone()
    again()
    x, graph, stream = xs[0].clone(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            y, a = block.step(x)
    torch.cuda.synchronize()
    for _ in range(2):
        again()
        for x_new, (y_want, a_want) in zip(xs, want):
            x.copy_(x_new)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, y_want) and torch.equal(a, a_want)
        assert torch.equal(block.cache.data, cache)


def test_the_example_runs(capsys):
    from attention_block import main

    say("4-bit attention block: the command")
    main(["--hidden", "512", "--head-dim", "64", "--kv-heads", "2", "--batch", "3", "--prompt", "90", "--steps", "4",
          "--bits", "4", "--rotary", "64"])
    assert "decode step" in capsys.readouterr().out
