"""Timed cases of the microscaled 4-bit linear and of the append to the 4-bit cache.

Microscaled 4-bit matrices (E2M1 elements, one power of two for every 32 along a
row) are what the matrix cores of gfx950 multiply directly.  The cases are the steps
of a program that holds its weights so: activations quantized by rows and by columns,
products of quantized matrices, the linear on 16-bit activations, both its
gradients; and new tokens of an attention layer, whose queries and keys are rotated
by their position while keys and values go into the paged FP4 cache.  ``run``
computes a case in plain torch operations (``own`` false) or with the package's
operators (``own`` true); ``exact`` computes the same outputs in 64 bits from the
definition.

A quantized [rows, k] matrix is codes uint8 [rows, kp / 2], element 2 j in the low
nibble of byte j, and scales uint8 [rows, kp / 32], kp = k rounded up to 128 and all
past k zeros: element = E2M1(code) * 2^(scale - 127).
"""

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- the cases -----------------------------------------------------------------

def _quantize(name, m, k, dtype, columns=False, wide=False):
    return {"name": name, "kind": "quantize", "m": m, "k": k, "dtype": dtype, "columns": columns, "wide": wide}


def _matmul(name, m, n, k, dtype, bias=False):
    return {"name": name, "kind": "matmul", "m": m, "n": n, "k": k, "dtype": dtype, "bias": bias}


def _linear(name, m, n, k, dtype, bias=False, wide=False):
    return {"name": name, "kind": "linear", "m": m, "n": n, "k": k, "dtype": dtype, "bias": bias, "wide": wide}


def _backward(name, m, n, k, dtype):
    return {"name": name, "kind": "backward", "m": m, "n": n, "k": k, "dtype": dtype}


def _append(name, tokens, heads, kv_heads, head_dim, rotary, page, dtype, runs=0, interleaved=False):
    return {"name": name, "kind": "append", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary": rotary, "page": page, "dtype": dtype, "runs": runs, "interleaved": interleaved}


def listed():
    return [
        # one token's activations of a 13B layer, quantized and read back: the smallest call
        _quantize("quantize_1x5120", 1, 5120, "f16"),
        # the activations of a 65B down projection
        _quantize("quantize_4096x22016_bf16", 4096, 22016, "bf16"),
        # an odd number of tokens of a 7B MLP by columns, as a weight's gradient takes them
        _quantize("quantize_cols_2047x11008", 2047, 11008, "f16", columns=True),
        # the first MLP layer of a small model, both sides quantized before, fp32 sums out
        _matmul("matmul_512x4096x1024_f32", 512, 4096, 1024, "f32"),
        # a 65B up projection of a prompt
        _matmul("matmul_4096x22016x8192", 4096, 22016, 8192, "f16"),
        # one token through a 13B up projection: a decode step
        _linear("linear_1x13824x5120", 1, 13824, 5120, "f16"),
        # sixteen sequences' tokens through a 13B down projection
        _linear("linear_16x5120x13824_bf16", 16, 5120, 13824, "bf16", bias=True),
        # a prompt through a 7B gate projection
        _linear("linear_2048x11008x4096", 2048, 11008, 4096, "f16"),
        # both gradients of a small model's MLP layer
        _backward("backward_512x4096x1024", 512, 4096, 1024, "f16"),
        # both gradients of a 7B projection
        _backward("backward_2048x4096x4096_bf16", 2048, 4096, 4096, "bf16"),
        # one token each of 64 sequences, grouped heads: a decode step
        _append("append_64_tokens_bf16", 64, 64, 8, 128, 128, 16, "bf16"),
        # a batch of prompts of 16000-odd tokens in all, 7B heads
        _append("append_prompts", 16381, 32, 32, 128, 128, 64, "f16", runs=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(("quantize", "matmul", "matmul", "linear", "linear", "linear", "backward", "append"))
    dtype = rng.choice(("f16", "bf16"))

    def width():  # of a layer: whole, or of any size
        return rng.choice((1024, 4096, 5120, 8192, 11008, 13824, 22016, _log(rng, 32, 22016), _log(rng, 32, 22016)))

    if kind == "append":
        head_dim = rng.choice((64, 128, 128, 256))
        heads, kv_heads = rng.choice(((16, 16), (32, 32), (40, 40), (64, 8), (28, 4), (8, 1), (6, 3)))
        most = 16381 * 96 * 128 // ((heads + 2 * kv_heads) * head_dim)
        c = _append("", _log(rng, 1, min(65536, most)), heads, kv_heads, head_dim,
                    rng.choice((head_dim, head_dim, head_dim // 2, head_dim // 4)), rng.choice((16, 32, 64, 128, 256)),
                    dtype, runs=rng.choice((0, 1, 3)), interleaved=rng.random() < 0.3)
    elif kind == "quantize":
        k = width()
        c = _quantize("", _log(rng, 1, min(16384, 4096 * 22016 // k)), k, dtype, columns=rng.random() < 0.4,
                      wide=rng.random() < 0.3)
    else:
        n, k = width(), width()
        if kind == "backward":
            most = 4096 * 8192 * 22016 // (2 * n * k)
            c = _backward("", _log(rng, 16, min(8192, most)), n, k, dtype)
        else:
            m = _log(rng, 1, min(8192, 4096 * 8192 * 22016 // (n * k)))
            if kind == "matmul":
                c = _matmul("", m, n, k, rng.choice(("f16", "bf16", "f32")), bias=rng.random() < 0.3)
            else:
                c = _linear("", m, n, k, dtype, bias=rng.random() < 0.5, wide=rng.random() < 0.3)
    del c["name"]
    return c


def work(case):
    kind = case["kind"]
    if kind == "append":
        t, q, kv, d = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
        token = kv * (d + 4 * (d // 64))  # cache bytes of one token
        # q, k and v in, q and the cache written, the cache read, the values it stands for out
        return {"bytes": t * (4 * q * d + 2 * token + 8 * kv * d + 24 + 4 * case["rotary"]),
                "flops": t * (3 * (q + kv) * case["rotary"] + 6 * kv * d)}
    m, k = case["m"], case["k"]
    held = lambda a, b: a * (-(-b // 2) + -(-b // 32))  # codes and scales
    if kind == "quantize":  # x in, codes and scales written and read, the values they stand for out
        a, b = (k, m) if case["columns"] else (m, k)
        return {"bytes": 4 * m * k + 2 * held(a, b), "flops": 3 * m * k}
    n = case["n"]
    if kind == "backward":
        return {"bytes": 2 * (m * n + 2 * m * k + 2 * n * k), "flops": 4 * m * n * k}
    out = 4 if case["dtype"] == "f32" else 2
    x = held(m, k) if kind == "matmul" else 2 * m * k
    return {"bytes": x + held(n, k) + out * (m * n + (n if case["bias"] else 0)), "flops": 2 * m * n * k}


# ---- the inputs ----------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, m, k, dtype, wide=False):
    """Activations with a few strong columns; with ``wide`` the columns of a wider matrix."""
    x = torch.empty((m, k + 48 if wide else k), dtype=dtype, device="cuda")
    strong = torch.where(torch.rand(x.shape[1], generator=gen, device="cuda") < 0.002, 20.0, 1.0)
    for i in range(0, m, 4096):
        x[i:i + 4096] = _normal(gen, min(4096, m - i), x.shape[1]) * strong
    if m > 8:
        x[m // 2] = 0  # a padded token
    return x[:, 16:16 + k] if wide else x


def _held(gen, rows, k, spread):
    """A quantized matrix: codes and scales as the module's docstring lays them out."""
    kp = -(-k // 128) * 128
    codes = torch.zeros((rows, kp // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((rows, kp // 32), dtype=torch.uint8, device="cuda")
    for i in range(0, rows, 4096):
        x = torch.zeros((min(4096, rows - i), kp), dtype=torch.float32, device="cuda")
        x[:, :k] = (_normal(gen, x.shape[0], k) * spread).half().float()
        c, e = _codes(x)
        codes[i:i + 4096] = c[:, 0::2] + 16 * c[:, 1::2]
        scales[i:i + 4096] = e
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    kind, dtype = case["kind"], DTYPES[case["dtype"]]
    state = {"case": dict(case), "dtype": dtype}
    if kind == "append":
        n, q, kv, d, page = (case[x] for x in ("tokens", "heads", "kv_heads", "head_dim", "page"))
        # runs of consecutive tokens that start inside a page (prompts), or one slot on a page of its own (decode)
        i = torch.arange(n, device="cuda")
        if case["runs"]:
            run = -(-n // case["runs"])
            at = i % run + 5 + i // run * (run + 5 + page)
            positions = i % run + 5
        else:
            at = i * page + torch.randint(0, page, (n,), generator=gen, device="cuda")
            positions = torch.randint(0, 131072, (n,), generator=gen, device="cuda")
        pages = int(at.max()) // page + 1
        order = torch.randperm(pages, generator=gen, device="cuda")
        slots = order[at // page] * page + at % page
        if n > 50:
            slots[n // 3] = -1  # padding: nothing is written, zeros are read
        x = _normal(gen, n, q + 2 * kv, d).to(dtype)  # as a projection leaves it
        half = case["rotary"] // 2
        rate = torch.exp2(-torch.arange(half, device="cuda", dtype=torch.float64) / half * math.log2(500000.0))
        angle = torch.arange(131072 if not case["runs"] else int(positions.max()) + 1, device="cuda")[:, None] * rate
        state.update(q=x[:, :q], k=x[:, q:q + kv], v=x[:, q + kv:], slots=slots, positions=positions,
                     cos=torch.cos(angle).float(), sin=torch.sin(angle).float(), page=page, head_dim=d,
                     data=torch.zeros((pages, kv, page * (d + 4 * (d // 64))), dtype=torch.uint8, device="cuda"))
        return state
    m, k = case["m"], case["k"]
    if kind == "quantize":
        state["x"] = _activations(gen, m, k, dtype, case["wide"])
        return state
    n = case["n"]
    if kind == "backward":
        state.update(x=_activations(gen, m, k, dtype), grad=(_normal(gen, m, n) * 0.01).to(dtype),
                     w=(_normal(gen, n, k) * 0.02).to(dtype))
        return state
    state["x"] = _held(gen, m, k, 1.0) if kind == "matmul" else _activations(gen, m, k, dtype, case["wide"])
    state.update(w=_held(gen, n, k, 0.02), k=k, bias=(_normal(gen, n) * 0.1).to(dtype) if case["bias"] else None)
    return state


# ---- the plain forms -------------------------------------------------------------

def _grid(f):
    """E2M1 magnitude codes of fp32 magnitudes: the nearest, ties to the even code, at most 6."""
    return ((f > 0.25).to(torch.uint8) + (f >= 0.75) + (f > 1.25) + (f >= 1.75) + (f > 2.5) + (f >= 3.5) + (f > 5.0))


def _codes(x):
    """(codes uint8, one each, and scales uint8 [rows, kp / 32]) of fp32 x [rows, kp]."""
    w = x.view(x.shape[0], -1, 32)
    e = (torch.frexp(w.abs().amax(-1)).exponent - 3).clamp(min=-127)  # floor(log2) - 2
    e = torch.where((w == 0).all(-1), -127, e)
    c = _grid(w.abs() * torch.exp2(-e.float())[..., None]) + 8 * torch.signbit(w).to(torch.uint8)
    return c.view(x.shape), (e + 127).to(torch.uint8)


def _rounded(x):
    """fp32 values that 16-bit x [rows, k] stands for once quantized."""
    rows, k = x.shape
    w = torch.zeros((rows, -(-k // 128) * 128), dtype=torch.float32, device=x.device)
    w[:, :k] = x
    return _values(*_codes(w))[:, :k]


def _values(codes, scales):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    v = lut[codes.int()].view(codes.shape[0], -1, 32) * torch.exp2(scales.float() - 127.0)[..., None]
    return v.view(codes.shape)


def _unheld(held):
    codes, scales = held
    return _values(torch.stack((codes & 15, codes >> 4), -1).flatten(-2), scales)


def _rotated(x, cos, sin, interleaved):
    """16-bit x [tokens, heads, D], the first dims of every head rotated: in 64 bits, since a
    value next to a border of the 4-bit grid decides a code; rounded to fp32, then to x's type."""
    r = 2 * cos.shape[-1]
    y = x[..., :r].double()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :r // 2], y[..., r // 2:])
    c, s = cos.double()[:, None], sin.double()[:, None]
    a, b = a * c - b * s, b * c + a * s
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y.float().to(x.dtype), x[..., r:]), -1)


def _cached(x):
    """The values that 16-bit x [..., D] stands for in the cache: blocks of 64 under their absmax."""
    w = x.float().unflatten(-1, (-1, 64))
    a = w.abs().amax(-1, keepdim=True)
    c = _grid(w.abs() * torch.where(a > 0, 6.0 * a.reciprocal(), 0.0))
    v = torch.tensor(E2M1, dtype=torch.float32, device=x.device)[c.int()] * (a / 6.0)
    return torch.where(torch.signbit(w), -v, v).flatten(-2).to(x.dtype)


def _plain(state):
    case, kind, dtype = state["case"], state["case"]["kind"], state["dtype"]
    if kind == "append":
        cos, sin = state["cos"][state["positions"]], state["sin"][state["positions"]]
        q, k = (_rotated(state[x], cos, sin, case["interleaved"]) for x in ("q", "k"))
        live = (state["slots"] >= 0)[:, None, None]
        return (q, *(torch.where(live, _cached(x), 0.0) for x in (k, state["v"])))
    if kind == "quantize":
        return _rounded(state["x"].t() if case["columns"] else state["x"]).to(dtype)
    if kind == "backward":
        g, x, w = state["grad"], state["x"], state["w"]
        grad_x = torch.matmul(_rounded(g), _rounded(w.t()).t())
        return grad_x.to(dtype), torch.matmul(_rounded(g.t()), _rounded(x.t()).t()).to(dtype)
    k = state["k"]
    x = _unheld(state["x"])[:, :k] if kind == "matmul" else _rounded(state["x"])
    out = torch.matmul(x, _unheld(state["w"])[:, :k].t())
    if state["bias"] is not None:
        out = out + state["bias"].float()
    return out.to(dtype)


def run(state):
    if not own:
        return _plain(state)
    import int8_mixed_precision_vectorwise_amd as i8
    case, kind, dtype = state["case"], state["case"]["kind"], state["dtype"]
    if kind == "append":
        cache = i8.Fp4Cache(state["data"], state["page"], state["head_dim"], dtype)
        q = i8.fp4_cache_append(cache, state["q"], state["k"], state["v"], state["slots"], state["positions"],
                                state["cos"], state["sin"], interleaved=case["interleaved"])
        return (q, *i8.fp4_cache_read(cache, state["slots"]))
    if kind == "quantize":
        return i8.mx4_dequantize(i8.mx4_quantize(state["x"], columns=case["columns"]), dtype)
    if kind == "backward":
        return i8.mx4_linear_backward(state["grad"], state["x"], state["w"])
    w = i8.Mx4Tensor(*state["w"], state["k"])
    if kind == "matmul":
        return i8.mx4_matmul(i8.Mx4Tensor(*state["x"], state["k"]), w, state["bias"], dtype)
    return i8.mx4_linear(state["x"], w, state["bias"])


# ---- the definition in 64 bits ----------------------------------------------------

def _exact_nearest(f):
    """The E2M1 magnitude nearest to float64 f >= 0; of two, the one with the even code; at most 6."""
    best, value = torch.full_like(f, math.inf), torch.zeros_like(f)
    for code, g in enumerate(E2M1):
        near = (f - g).abs()
        better = (near < best) | ((near == best) & (code % 2 == 0))
        best, value = torch.where(better, near, best), torch.where(better, torch.full_like(f, g), value)
    return value


def _exact_rounded(x):
    """float64 values of x [rows, k] quantized in blocks of 32 along its rows."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // x.shape[1])
    for i in range(0, x.shape[0], step):
        w = torch.nn.functional.pad(x[i:i + step].double(), (0, -x.shape[1] % 32)).unflatten(1, (-1, 32))
        top = w.abs().max(-1, keepdim=True).values
        scale = torch.exp2((torch.floor(torch.log2(top)) - 2).clamp(min=-127.0))
        v = _exact_nearest(w.abs() / scale) * scale
        out[i:i + step] = torch.where(w < 0, -v, v).flatten(1)[:, :x.shape[1]]
    return out


def _exact_held(held, k):
    """float64 values of codes and scales, from the bits."""
    codes, scales = held
    j = torch.arange(k, device=codes.device)
    code = (codes[:, j // 2].int() >> (4 * (j % 2)).int()) & 15
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    return torch.where(code > 7, -mag, mag) * torch.exp2(scales[:, j // 32].double() - 127)


def _exact_rotated(x, cos, sin, interleaved):
    """float64 [tokens, heads, D], every pair turned as one complex number."""
    half, out = cos.shape[-1], x.double()
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    turned = torch.complex(out[..., first], out[..., second]) * torch.complex(cos.double(), sin.double())[:, None]
    out[..., first], out[..., second] = turned.real, turned.imag
    return out


def _exact_cached(x):
    """float64 values of 16-bit x [..., D] in the cache; a code is decided in binary32, as defined."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for b in range(0, x.shape[-1], 64):
        w = x[..., b:b + 64].float()
        a = w.abs().max(-1, keepdim=True).values
        f = torch.where(a > 0, w.abs() * (6.0 * (1.0 / a)), torch.zeros_like(w)).double()
        v = _exact_nearest(f) * a.double() / 6
        out[..., b:b + 64] = torch.where(w < 0, -v, v)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "append":
        n, parts = case["tokens"], ([], [], [])
        for i in range(0, n, 2048):
            at = slice(i, i + 2048)
            cos, sin = (state[t][state["positions"][at]] for t in ("cos", "sin"))
            q, k = (_exact_rotated(state[x][at], cos, sin, case["interleaved"]) for x in ("q", "k"))
            live = (state["slots"][at] >= 0)[:, None, None]
            parts[0].append(q)
            # the cache takes keys in its own type
            for part, x in ((1, k.float().to(state["dtype"])), (2, state["v"][at])):
                parts[part].append(torch.where(live, _exact_cached(x), 0.0))
        return tuple(torch.cat(p) for p in parts)
    if kind == "quantize":
        return _exact_rounded(state["x"].t().contiguous() if case["columns"] else state["x"])
    if kind == "backward":
        g, x, w = state["grad"], state["x"], state["w"]
        by_columns = lambda t: _exact_rounded(t.t().contiguous())
        return _exact_rounded(g) @ by_columns(w).t(), by_columns(g) @ by_columns(x).t()
    k = case["k"]
    x = _exact_held(state["x"], k) if kind == "matmul" else _exact_rounded(state["x"])
    out = x @ _exact_held(state["w"], k).t()
    return out if state["bias"] is None else out + state["bias"].double()
