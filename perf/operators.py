"""Timed cases of the 4-bit key/value cache operators: write, read back, attention.

Each case names one call of a serving program: new keys and values are
quantized into a paged FP4 (E2M1) cache as they are written, slots are read
back as 16-bit values, and queries (one token a sequence, a few, or a whole
prompt) attend over the cache.  ``run`` computes a case in plain torch
operations in fp32 (``own`` false) or with the package's operators (``own``
true); ``exact`` computes the same outputs in 64 bits from the definition.

The cache is uint8 [pages, kv_heads, slab].  A slab holds one page of one head,
P tokens of D = 64 NB dimensions, in four parts:

* K codes, per token 32 NB bytes: [4 groups g][NB blocks b][8 bytes], the bytes
  holding dimensions 64 b + 16 g + (0..15), the even one in the low nibble;
* V codes, per 4 tokens 128 NB bytes: [16 groups m][NB blocks b][4 tokens in the
  order 0, 2, 1, 3][2 bytes], the bytes holding dimensions 64 b + 4 m + (0..3);
* K scales, then V scales: [P tokens][NB blocks], each the block's absmax in the
  cache's 16-bit type.
"""

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---- the cases -----------------------------------------------------------------

def _move(name, kind, tokens, kv_heads, head_dim, page, dtype, runs=0):
    return {"name": name, "kind": kind, "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "dtype": dtype, "runs": runs}


def _attend(name, batch, q_len, past, kv_heads, group, head_dim, page, dtype, ragged=False, window=0, softcap=0.0,
            alibi=False, prefix=0):
    return {"name": name, "kind": "attend", "batch": batch, "q_len": q_len, "past": past, "kv_heads": kv_heads,
            "group": group, "head_dim": head_dim, "page": page, "dtype": dtype, "ragged": ragged, "window": window,
            "softcap": softcap, "alibi": alibi, "prefix": prefix}


def listed():
    return [
        # one token of one sequence, 13B heads: the smallest call of a decode step
        _move("write_1_token", "write", 1, 40, 128, 64, "f16"),
        # one token each of 64 sequences, grouped heads
        _move("write_64_tokens_bf16", "write", 64, 8, 128, 16, "bf16"),
        # a batch of prompts of 16000-odd tokens in all, 7B heads
        _move("write_prompts", "write", 16381, 32, 128, 64, "f16", runs=4),
        # a prompt of a small model read back, odd length
        _move("read_1001_tokens", "read", 1001, 16, 64, 16, "f16", runs=1),
        # a long context read back (to leave the cache for another type or place)
        _move("read_65536_tokens", "read", 65536, 8, 128, 128, "bf16", runs=1),
        # a decode step of a small model, one short sequence: latency
        _attend("decode_b1_small", 1, 1, 128, 16, 1, 64, 16, "f16"),
        # a decode step of a 13B model, 16 sequences of different lengths, one slot idle, distance bias
        _attend("decode_b16_alibi", 16, 1, 2047, 40, 1, 128, 64, "f16", ragged=True, alibi=True),
        # a decode step of 64 long sequences, grouped heads
        _attend("decode_b64_grouped", 64, 1, 8191, 8, 8, 128, 64, "bf16", ragged=True),
        # one very long sequence: the work of a few heads split over the chip
        _attend("decode_b1_131072", 1, 1, 131071, 8, 8, 128, 128, "f16"),
        # four drafted tokens a sequence, capped scores, a window past the first tokens, wide heads
        _attend("draft_window_softcap", 8, 4, 4000, 4, 4, 256, 32, "f16", ragged=True, window=1024, softcap=50.0, prefix=4),
        # pieces of prompts behind what is cached already, different lengths
        _attend("prompt_pieces", 6, 700, 3001, 8, 4, 128, 64, "bf16", ragged=True, softcap=30.0),
        # a whole prompt of a 65B model
        _attend("prompt_4096", 1, 4096, 0, 64, 1, 128, 64, "f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(("write", "read", "decode", "decode", "draft", "prompt"))
    dtype = rng.choice(("f16", "bf16"))
    head_dim = rng.choice((64, 128, 128, 256))
    page = rng.choice((16, 32, 64, 128, 256))
    if kind in ("write", "read"):
        heads = rng.choice((1, 2, 4, 8, 16, 32, 40))
        most = 16381 * 32 * 128 // (heads * head_dim)
        c = _move("", kind, _log(rng, 1, min(65536, most)), heads, head_dim, page, dtype, rng.choice((0, 1, 3)))
    else:
        heads, group = rng.choice(((16, 1), (32, 1), (40, 1), (8, 8), (8, 4), (4, 7), (2, 16), (1, 32), (3, 2)))
        if kind == "prompt":
            q_len = _log(rng, 17, 4096)
            past = rng.choice((0, _log(rng, 1, 4096)))
            batch = _log(rng, 1, 16)
            most = 64 * 4096 * 4096 // 2
        else:
            q_len = 1 if kind == "decode" else rng.randint(2, 12)
            past = _log(rng, 1, 131071)
            batch = _log(rng, 1, 128)
            most = 1 << 40
        # no dearer than the largest listed case, padded to the longest sequence
        while (batch > 1 and (batch * heads * group * q_len * (past + q_len) > most
                              or batch * heads * head_dim * (past + q_len) > 64 * 8192 * 8 * 128)):
            batch -= 1
        while (heads * group * q_len * (past + q_len) > most or heads * head_dim * (past + q_len) > 64 * 8192 * 8 * 128):
            q_len, past = (max(17, q_len // 2), past // 2) if kind == "prompt" else (q_len, past // 2)
        c = _attend("", batch, q_len, past, heads, group, head_dim, page, dtype, ragged=rng.random() < 0.6,
                    window=rng.choice((0, 0, _log(rng, 1, 4096))), softcap=rng.choice((0.0, 0.0, 30.0)),
                    alibi=rng.random() < 0.3, prefix=rng.choice((0, 0, rng.randint(1, 200))))
    del c["name"]
    return c


def _lengths(case):
    """(query tokens, cached tokens ahead of them) of every sequence; the first has the most."""
    r = random.Random(case["batch"] * 1000003 + case["past"])
    q, past = [case["q_len"]], [case["past"]]
    for _ in range(case["batch"] - 1):
        q.append(1 + int((case["q_len"] - 1) * r.random()) if case["ragged"] else case["q_len"])
        past.append(int(case["past"] * (0.25 + 0.75 * r.random())) if case["ragged"] else case["past"])
    if case["ragged"] and case["batch"] >= 8:
        past[-1] = -q[-1]  # an idle slot of the batch: no tokens at all, its rows see nothing
    return q, past


def work(case):
    d, heads = case["head_dim"], case["kv_heads"]
    token = heads * (d + 4 * (d // 64))  # cache bytes of one token
    if case["kind"] == "read":
        return {"bytes": case["tokens"] * (token + 4 * heads * d + 8), "flops": 2 * case["tokens"] * heads * d}
    if case["kind"] == "write":  # k and v in, the cache written and read, the values it stands for out
        return {"bytes": case["tokens"] * (2 * token + 8 * heads * d + 16), "flops": 6 * case["tokens"] * heads * d}
    q_heads, window, pairs, tokens = heads * case["group"], case["window"] or 1 << 40, 0, 0
    lens = list(zip(*_lengths(case)))
    for q, past in lens:
        length = past + q
        if length <= 0:
            continue
        fixed = min(case["prefix"], length)
        for p in range(past, length):
            low = max(0, p + 1 - window)
            pairs += p + 1 - low + min(fixed, low) + max(0, fixed - p - 1)
        low = max(0, past + 1 - window)
        tokens += length - low + min(fixed, low)
    rows = sum(q for q, _ in lens)
    table = sum(-(-max(q + past, 0) // case["page"]) for q, past in lens)
    return {"bytes": rows * q_heads * (4 * d + 4) + tokens * token + 4 * table, "flops": 4 * pairs * q_heads * d}


# ---- the inputs ----------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys_values(gen, tokens, heads, d, dtype):
    """Keys with a few strong dimensions, values of a spread of magnitudes."""
    strong = torch.where(torch.rand((heads, d), generator=gen, device="cuda") < 0.03, 6.0, 1.0)
    k = _normal(gen, tokens, heads, d) * strong
    v = _normal(gen, tokens, heads, d) * torch.exp(_normal(gen, tokens, 1, 1) * 0.5)
    return k.to(dtype), v.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dtype, heads, d, page = DTYPES[case["dtype"]], case["kv_heads"], case["head_dim"], case["page"]
    state = {"case": dict(case), "page": page, "head_dim": d, "dtype": dtype}
    slab = page * (d + 4 * (d // 64))
    if case["kind"] != "attend":
        n, runs = case["tokens"], case["runs"]
        # runs of consecutive tokens that start inside a page (prompts), or one slot on a page of its own (decode)
        if runs:
            run = -(-n // runs)
            i = torch.arange(n, device="cuda")
            at = i % run + 5 + i // run * (run + 5 + page)
        else:
            at = torch.arange(n, device="cuda") * page + torch.randint(0, page, (n,), generator=gen, device="cuda")
        pages = int(at.max()) // page + 1
        order = torch.randperm(pages, generator=gen, device="cuda")
        slots = order[at // page] * page + at % page
        if n > 50:
            slots[n // 3] = -1  # padding: nothing is written, zeros are read
        k, v = _keys_values(gen, n, heads, d, dtype)
        data = torch.zeros((pages, heads, slab), dtype=torch.uint8, device="cuda")
        state.update(slots=slots, data=data)
        if case["kind"] == "write":
            state.update(k=k, v=v)
        else:
            _plain_write(state, k, v)
        return state
    q_len, past = _lengths(case)
    length = [a + b for a, b in zip(q_len, past)]
    cols = max(1, -(-max(length) // page))
    used = [-(-n // page) for n in length]
    order = torch.randperm(max(1, sum(used)), generator=gen, device="cuda")
    table = torch.zeros((case["batch"], cols), dtype=torch.int64, device="cuda")
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    data = torch.empty((order.numel(), heads, slab), dtype=torch.uint8, device="cuda")
    state["data"] = data
    for p in range(0, order.numel(), max(1, (1 << 26) // (page * heads * d))):
        n = min(order.numel(), p + max(1, (1 << 26) // (page * heads * d))) - p
        k, v = _keys_values(gen, n * page, heads, d, dtype)
        state["slots"] = torch.arange(p * page, (p + n) * page, device="cuda")
        _plain_write(state, k, v)
    del state["slots"]
    # slots past a sequence's end hold what was there before: scales that are no numbers, among others
    scales = data.view(torch.int16)[:, :, page * d // 2:].view(order.numel(), heads, 2, page, d // 64)
    for i, n in enumerate(length):
        if n % page:
            scales[table[i, n // page], :, :, n % page:] = 0x7fff
    rows = sum(q_len)
    state.update(
        q=(_normal(gen, rows, heads * case["group"], d) * 1.5).to(dtype),
        table=table.to(torch.int32),
        lengths=torch.tensor(length, dtype=torch.int32, device="cuda"),
        q_offsets=torch.tensor([sum(q_len[:i]) for i in range(len(q_len) + 1)], dtype=torch.int32, device="cuda")
        if case["ragged"] else None,
        max_q=max(q_len),
        alibi=torch.exp2(-8.0 * torch.arange(1, heads * case["group"] + 1, device="cuda") / (heads * case["group"]))
        if case["alibi"] else None,
        prefix=torch.full((case["batch"],), case["prefix"], dtype=torch.int32, device="cuda") if case["prefix"] else None)
    return state


# ---- the plain forms -------------------------------------------------------------

def _scale_bytes(a, dtype):
    return a.to(dtype).view(torch.uint8)  # the absmax of 16-bit numbers is one of them: nothing is rounded


def _encode(x):
    """(codes uint8, one each, and absmax fp32 [..., NB]) of 16-bit x [..., D], blocks of 64."""
    w = x.float().unflatten(-1, (-1, 64))
    a = w.abs().amax(-1)
    inv = torch.where(a > 0, 6.0 / a, 0.0)
    f = w.abs() * inv[..., None]
    mag = ((f > 0.25).to(torch.uint8) + (f >= 0.75) + (f > 1.25) + (f >= 1.75) + (f > 2.5) + (f >= 3.5) + (f > 5.0))
    return (mag + 8 * torch.signbit(w).to(torch.uint8)).flatten(-2), a


def _places(state, slots):
    """First byte of each (slot, head) in the flat cache, and the token's place in its page."""
    heads, slab = state["data"].shape[1:]
    page = torch.div(slots, state["page"], rounding_mode="floor")
    return (page[:, None] * heads + torch.arange(heads, device=slots.device)) * slab, slots % state["page"]


def _addresses(state, slots):
    """Byte addresses of each (slot, head): K codes, V codes, K scales, V scales."""
    d, page = state["head_dim"], state["page"]
    nb = d // 64
    base, t = _places(state, slots)
    dev = slots.device
    k = base[..., None] + (t * (d // 2))[:, None, None] + torch.arange(d // 2, device=dev)
    pair = torch.arange(16 * nb, device=dev)[:, None] * 8 + torch.arange(2, device=dev)
    place = (t % 4 % 2) * 2 + t % 4 // 2  # tokens 0, 1, 2, 3 of a group lie at 0, 2, 1, 3
    v = (base[..., None, None] + page * d // 2 + (t // 4 * (2 * d) + place * 2)[:, None, None, None] + pair).flatten(-2)
    s = base[..., None] + page * d + (t * 2 * nb)[:, None, None] + torch.arange(2 * nb, device=dev)
    return k, v, s, s + page * 2 * nb


def _plain_write(state, k, v):
    nb, heads = state["head_dim"] // 64, k.shape[1]
    keep = state["slots"] >= 0
    slots, k, v = state["slots"][keep], k[keep], v[keep]
    flat = state["data"].view(-1)
    ak, av, ask, asv = _addresses(state, slots)
    (ck, sk), (cv, sv) = _encode(k), _encode(v)
    ck, cv = ck[..., 0::2] + 16 * ck[..., 1::2], cv[..., 0::2] + 16 * cv[..., 1::2]
    n = slots.numel()
    flat[ak] = ck.view(n, heads, nb, 4, 8).transpose(2, 3).reshape(n, heads, -1)
    flat[av] = cv.view(n, heads, nb, 16, 2).transpose(2, 3).reshape(n, heads, -1)
    flat[ask] = _scale_bytes(sk, state["dtype"])
    flat[asv] = _scale_bytes(sv, state["dtype"])


def _values(codes, absmax):
    """fp32 values of one-byte codes [..., NB, 64] under block absmax [..., NB]."""
    lut = torch.tensor(E2M1, dtype=torch.float32, device=codes.device)
    return (lut[codes.int()] * (absmax.float() / 6.0)[..., None]).flatten(-2)


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _plain_read(state):
    nb, heads = state["head_dim"] // 64, state["data"].shape[1]
    slots = state["slots"]
    live = (slots >= 0)[:, None, None]
    flat = state["data"].view(-1)
    ak, av, ask, asv = _addresses(state, slots.clamp(min=0))
    n, dtype = slots.numel(), state["dtype"]
    ck = _nibbles(flat[ak].view(n, heads, 4, nb, 8)).transpose(2, 3).reshape(n, heads, nb, 64)
    cv = _nibbles(flat[av].view(n, heads, 16, nb, 2)).transpose(2, 3).reshape(n, heads, nb, 64)
    return tuple(torch.where(live, _values(c, flat[a].view(dtype)), 0.0).to(dtype) for c, a in ((ck, ask), (cv, asv)))


def _gather(state):
    """Keys and values fp32 [batch, heads, tokens, D] of every sequence, whole pages."""
    page, d = state["page"], state["head_dim"]
    nb, heads = d // 64, state["data"].shape[1]
    slabs = state["data"][state["table"].long()].transpose(1, 2)  # [batch, heads, pages, slab]
    lead, half = slabs.shape[:3], page * d // 2
    ck = _nibbles(slabs[..., :half].reshape(*lead, page, 4, nb, 8)).transpose(4, 5).reshape(*lead, page, nb, 64)
    cv = _nibbles(slabs[..., half:2 * half].reshape(*lead, page // 4, 16, nb, 4, 2))
    cv = cv[..., (0, 2, 1, 3), :].permute(0, 1, 2, 3, 6, 5, 4, 7).reshape(*lead, page, nb, 64)
    scales = slabs[..., 2 * half:].contiguous().view(state["dtype"]).view(*lead, 2, page, nb)
    return tuple(_values(c, scales[..., i, :, :]).reshape(*lead[:2], -1, d) for i, c in enumerate((ck, cv)))


def _plain_attend(state):
    c, q, dev = state["case"], state["q"], state["q"].device
    heads, group, d, top = c["kv_heads"], c["group"], c["head_dim"], state["max_q"]
    batch = c["batch"]
    lengths = state["lengths"].long()
    off = state["q_offsets"].long() if state["q_offsets"] is not None else torch.arange(batch + 1, device=dev) * top
    q_len = off[1:] - off[:-1]
    i = torch.arange(top, device=dev)
    rows = (off[:-1, None] + i).clamp(max=q.shape[0] - 1)  # [batch, max_q], the rest is padding
    k, v = _gather(state)
    j = torch.arange(k.shape[2], device=dev)
    inside = j < lengths[:, None]
    k = torch.where(inside[:, None, :, None], k, 0.0)
    v = torch.where(inside[:, None, :, None], v, 0.0)
    qp = q[rows].float().view(batch, top, heads, group, d).permute(0, 2, 3, 1, 4).reshape(batch, heads, group * top, d)
    s = (torch.matmul(qp, k.transpose(2, 3)) / math.sqrt(d)).view(batch, heads, group, top, -1)
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    p = (lengths - q_len)[:, None] + i  # positions [batch, max_q]
    away = p[:, :, None] - j
    if state["alibi"] is not None:
        s = s - state["alibi"].view(1, heads, group, 1, 1) * away.abs()[:, None, None].float()
    see = away >= 0
    if c["window"]:
        see &= away < c["window"]
    if state["prefix"] is not None:
        see |= j < state["prefix"].long()[:, None, None]
    see &= inside[:, None] & (p >= 0)[:, :, None]
    s = torch.where(see[:, None, None], s, -math.inf)
    top_s = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top_s == -math.inf, 0.0, top_s))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(batch, heads, group * top, -1), v).view(batch, heads, group, top, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top_s + torch.log(total)).squeeze(-1)
    at = (i < q_len[:, None])
    out = o.permute(0, 3, 1, 2, 4)[at].reshape(q.shape).to(q.dtype)
    return out, lse.permute(0, 3, 1, 2)[at].reshape(q.shape[:2])


def run(state):
    kind = state["case"]["kind"]
    if own:
        import int8_mixed_precision_vectorwise_amd as i8
        cache = i8.Fp4Cache(state["data"], state["page"], state["head_dim"], state["dtype"])
        if kind == "attend":
            c = state["case"]
            return i8.fp4_cache_attention(state["q"], cache, state["table"], state["lengths"],
                                          q_offsets=state["q_offsets"], max_q=state["max_q"], window=c["window"],
                                          softcap=c["softcap"], alibi=state["alibi"], prefix=state["prefix"],
                                          return_lse=True)
        if kind == "write":
            i8.fp4_cache_write(cache, state["k"], state["v"], state["slots"])
        return i8.fp4_cache_read(cache, state["slots"])
    if kind == "attend":
        return _plain_attend(state)
    if kind == "write":
        _plain_write(state, state["k"], state["v"])
    return _plain_read(state)


# ---- the definition in 64 bits ----------------------------------------------------

def _exact_quantized(x):
    """The values that 16-bit x [..., D] stands for once quantized; a code is decided in binary32, as defined."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    grid = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    for b in range(0, x.shape[-1], 64):
        w = x[..., b:b + 64].float()
        a = w.abs().max(-1, keepdim=True).values
        f = torch.where(a > 0, w.abs() * (6.0 / a), torch.zeros_like(w)).double()
        best, value = torch.full_like(f, math.inf), torch.zeros_like(f)
        for code, g in enumerate(grid):  # the nearest; of two, the even code
            near = (f - g).abs()
            better = (near < best) | ((near == best) & (code % 2 == 0))
            best, value = torch.where(better, near, best), torch.where(better, torch.full_like(f, g), value)
        out[..., b:b + 64] = torch.where(w < 0, -value, value) * a.double() / 6
    return out


def _exact_cached(state, slots, values):
    """float64 [slots, heads, D] of the keys or values held at the slots, byte by byte from the layout."""
    data, P, D = state["data"].reshape(-1), state["page"], state["head_dim"]
    heads, slab = state["data"].shape[1:]
    nb, dev = D // 64, slots.device
    d = torch.arange(D, device=dev)
    b, r = d // 64, d % 64
    page, t = slots // P, slots % P
    first = (page[:, None] * heads + torch.arange(heads, device=dev)[None, :])[:, :, None] * slab
    if values:
        place = torch.tensor([0, 2, 1, 3], device=dev)[t % 4]
        byte = P * 32 * nb + (t // 4 * 128 * nb + place * 2)[:, None] + (r // 4 * 8 * nb + b * 8 + r % 4 // 2)[None, :]
    else:
        byte = (t * 32 * nb)[:, None] + (r // 16 * 8 * nb + b * 8 + r % 16 // 2)[None, :]
    code = (data[first + byte[:, None, :]] >> (4 * (d % 2)).to(torch.uint8)) & 15
    e, m = ((code >> 1) & 3).double(), (code & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
    at = first + (P * 64 * nb + (P * 2 * nb if values else 0) + (t[:, None] * nb + b[None, :]) * 2)[:, None, :]
    bits = data[at].to(torch.int32) + data[at + 1].to(torch.int32) * 256
    a = (bits - 65536 * (bits > 32767)).to(torch.int16).view(state["dtype"]).double()
    return torch.where(code > 7, -mag, mag) * a / 6


def exact(case, seed):
    state = prepare(case, seed)
    if case["kind"] == "write":
        live = (state["slots"] >= 0)[:, None, None]
        return tuple(torch.cat([torch.where(live[i:i + 4096], _exact_quantized(x[i:i + 4096]), 0.0)
                                for i in range(0, x.shape[0], 4096)]) for x in (state["k"], state["v"]))
    if case["kind"] == "read":
        slots = state["slots"]
        live = (slots >= 0)[:, None, None]
        return tuple(torch.cat([torch.where(live[i:i + 4096], _exact_cached(state, slots[i:i + 4096].clamp(min=0), x), 0.0)
                                for i in range(0, slots.numel(), 4096)]) for x in (False, True))
    q, dev = state["q"], state["q"].device
    heads, group, D = case["kv_heads"], case["group"], case["head_dim"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=dev)
    row = 0
    for n, (q_len, past) in enumerate(zip(*_lengths(case))):
        length, rows = past + q_len, slice(row, row + q_len)
        row += q_len
        if length <= 0:
            continue
        j = torch.arange(length, device=dev)
        slots = state["table"][n].long()[j // case["page"]] * case["page"] + j % case["page"]
        k, v = (torch.cat([_exact_cached(state, slots[i:i + 8192], x) for i in range(0, length, 8192)]) for x in (False, True))
        p = torch.arange(past, length, device=dev)[:, None]
        see = (j <= p) & (j > p - (case["window"] or length + 1)) | (j < case["prefix"])
        for h in range(heads * group):
            s = q[rows, h].double() @ k[:, h // group].t().contiguous() / D ** 0.5
            if case["softcap"]:
                s = torch.tanh(s / case["softcap"]) * case["softcap"]
            if case["alibi"]:
                s = s - state["alibi"][h].double() * (p - j).abs()
            s = s.masked_fill(~see, -math.inf)
            lse[rows, h] = torch.logsumexp(s, -1)
            out[rows, h] = torch.softmax(s, -1) @ v[:, h // group].contiguous()
    return out, lse
