"""An attention block that serves: quantized projections around a 4-bit key/value cache.

One layer's path, for prompts of different lengths and then token by token:

    x -> linear -> q, k, v -> fp4_cache_write -> fp4_cache_attention -> linear

with int8 weights, or microscaled 4-bit weights and activations; with positions,
fp4_cache_append rotates q in place and k on its way into the cache.  k and v are
written from where the projection left them (views of its output); the cache, the page
table and the lengths stay on the device, so that a decode step is a fixed sequence of
launches and can be captured into a HIP graph.

    python examples/attention_block.py            # sizes of a 13B layer, 16 sequences
    python examples/attention_block.py --hidden 4096 --kv-heads 8 --batch 64 --prompt 4000
    python examples/attention_block.py --bits 4 --rotary 128
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int8_mixed_precision_vectorwise_amd as i8  # noqa: E402


class AttentionBlock:
    """Projections with weights of ``bits`` (8 or 4) and the cache of ``batch`` sequences of up to ``max_len`` tokens,
    whose positions turn the first ``rotary`` dims of a head (0: none)."""

    def __init__(self, w_qkv, w_out, heads, kv_heads, batch, max_len, page_size=64, window=0, bits=8, rotary=0):
        dev = w_qkv.device
        self.head_dim = w_out.shape[1] // heads
        self.heads, self.kv_heads, self.window = heads, kv_heads, window
        if bits == 4:
            self.linear, self.qkv, self.out = i8.mx4_linear, (i8.mx4_quantize(w_qkv),), (i8.mx4_quantize(w_out),)
        else:
            self.linear, self.qkv, self.out = i8.linear, i8.quantize_weight(w_qkv), i8.quantize_weight(w_out)
        cols = -(-max_len // page_size)
        self.cache = i8.Fp4Cache.create(batch * cols, kv_heads, self.head_dim, page_size, w_qkv.dtype, dev)
        # any order of pages will do; a server hands them out as sequences grow
        self.table = torch.randperm(batch * cols, device=dev).to(torch.int32).view(batch, cols)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.rotary, self.place = rotary, None
        if rotary:
            rate = 10000.0 ** (-torch.arange(0, rotary, 2, device=dev, dtype=torch.float64) / rotary)
            angle = torch.arange(cols * page_size, device=dev)[:, None] * rate
            self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def slots(self, seq, place):
        """Cache slots of tokens at ``place`` of sequences ``seq`` (int64 each)."""
        page = self.cache.page_size
        return self.table[seq, place // page].long() * page + place % page

    def attend(self, x, slots, q_offsets, max_q):
        """The block on x [tokens, hidden], at self.place of their sequences, whose tokens the lengths already count:
        (y, attention's output)."""
        y = self.linear(x, *self.qkv).view(x.shape[0], self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], 1)
        if self.rotary:
            i8.fp4_cache_append(self.cache, q, k, v, slots, self.place, self.cos, self.sin, out=q)
        else:
            i8.fp4_cache_write(self.cache, k, v, slots)
        a = i8.fp4_cache_attention(q, self.cache, self.table, self.lengths, q_offsets, max_q, window=self.window)
        return self.linear(a.view(x.shape[0], -1), *self.out), a

    def prompt(self, x, counts):
        """New tokens of every sequence, counts[b] of them in order, behind what it has (0: none)."""
        dev = x.device
        n = torch.tensor(counts, device=dev)
        seq = torch.repeat_interleave(torch.arange(len(counts), device=dev), n)
        offsets = torch.cat((n.new_zeros(1), n.cumsum(0)))
        self.place = self.lengths.long()[seq] + torch.arange(len(seq), device=dev) - offsets[seq]
        self.lengths += n.to(torch.int32)
        return self.attend(x, self.slots(seq, self.place), offsets.to(torch.int32), max(counts))

    def step(self, x):
        """One new token of every sequence; launches only, no copy to the host."""
        self.place = self.lengths.long()
        slots = self.slots(torch.arange(x.shape[0], device=x.device), self.place)
        self.lengths += 1
        return self.attend(x, slots, None, 1)


def timed(f, steps):
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    f()
    start.record()
    for _ in range(steps):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / steps * 1e3


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--hidden", type=int, default=5120)
    p.add_argument("--head-dim", type=int, default=128)
    p.add_argument("--kv-heads", type=int, default=0, help="0: as many as query heads")
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--prompt", type=int, default=1000, help="longest prompt; the others are shorter")
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--bits", type=int, choices=(8, 4), default=8, help="of the projections' weights")
    p.add_argument("--rotary", type=int, default=0, help="dims of a head that turn by position")
    o = p.parse_args(argv)
    torch.manual_seed(0)
    heads = o.hidden // o.head_dim
    kv_heads = o.kv_heads or heads
    rows = (heads + 2 * kv_heads) * o.head_dim
    w_qkv = (torch.randn(rows, o.hidden, device="cuda") * o.hidden ** -0.5).half()
    w_out = (torch.randn(o.hidden, heads * o.head_dim, device="cuda") * o.hidden ** -0.5).half()
    block = AttentionBlock(w_qkv, w_out, heads, kv_heads, o.batch, o.prompt + 2 * o.steps + 8, window=o.window,
                           bits=o.bits, rotary=o.rotary)
    counts = [max(1, o.prompt - o.prompt * i // (2 * o.batch)) for i in range(o.batch)]
    y, _ = block.prompt(torch.randn(sum(counts), o.hidden, device="cuda").half(), counts)
    x = y[torch.tensor(counts, device="cuda").cumsum(0) - 1].contiguous()
    eager = timed(lambda: block.step(x), o.steps)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            y, _ = block.step(x)
    torch.cuda.synchronize()
    replay = timed(graph.replay, o.steps - 1)
    mib = block.cache.data.numel() / 2 ** 20
    print(f"hidden {o.hidden}, {heads} / {kv_heads} heads of {o.head_dim}, {o.batch} sequences of "
          f"{int(block.lengths.min())} to {int(block.lengths.max())} tokens: decode step {eager:.1f} us, "
          f"{replay:.1f} us from a graph; cache {mib:.0f} MiB ({mib * 64 / 17:.0f} in 16 bits)")


if __name__ == "__main__":
    main()
