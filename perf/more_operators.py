"""Measured cases of rotary positions, of the paged append that applies them, and of attention with dropout.

``listed()`` names the cases, ``prepare()`` makes one case's inputs on the GPU,
``run()`` does one pass, ``work()`` says what a pass cannot do without, and
``exact()`` gives the outputs in 64 bits.  With ``own`` false, ``run()``
computes the plain form (elementary torch operations); with ``own`` true it
makes the package's calls.

Rotary positions: element pair i of the first ``rot`` elements of a row turns by
position * freqs[i] (fractions of a turn, held as 64-bit integers in units of
2^-64 turn), times an amplitude.  Dropout: element (b, h, i, j) of the softmax is
kept where an 8-bit number u, from bit j % 32 of the eight words that
Philox4x32 with seven rounds gives for (i, 2 * (j // 32) + {0, 1}, b * Hq + h, offset) under
the key ``seed``, is at least T = round(256 * p), and divided by 1 - T / 256.
"""
import math
import random

import torch

own = False

PAGES = (16, 32, 64, 128)
HEADS = ((32, 8), (16, 16), (8, 2), (16, 1), (6, 2), (32, 32))
SCALING = ("none", "linear", "parts")
M32 = 0xFFFFFFFF


def _pkg():
    import exact_attention_95_gb300 as pkg
    return pkg


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decoding step of 64 requests: queries and keys are slices of a
        # packed projection, at positions far into their contexts.
        {"name": "rope-decode-64", "op": "rope", "bwd": False, "layout": "tokens", "B": 1, "N": 64, "Hq": 32, "Hkv": 8,
         "d": 128, "rot": 128, "interleaved": False, "dtype": "bf16", "scaling": "parts", "far": 131072},
        # The benchmark's layer in training: out of the packed projection into
        # the layout that the attention reads.
        {"name": "rope-packed-4096", "op": "rope", "bwd": False, "layout": "packed", "B": 2, "N": 4096, "Hq": 32,
         "Hkv": 32, "d": 128, "rot": 128, "interleaved": False, "dtype": "bf16", "scaling": "none", "far": 0},
        # Gradients of that layer's queries and keys back into the packed gradient.
        {"name": "rope-bwd-4096", "op": "rope", "bwd": True, "layout": "packed", "B": 2, "N": 4096, "Hq": 32, "Hkv": 32,
         "d": 128, "rot": 128, "interleaved": False, "dtype": "bf16", "scaling": "none", "far": 0},
        # Gradients where half of each head turns, adjacent elements paired, in
        # 32 bits, ragged.
        {"name": "rope-bwd-1001-f32", "op": "rope", "bwd": True, "layout": "heads", "B": 3, "N": 1001, "Hq": 16,
         "Hkv": 4, "d": 64, "rot": 32, "interleaved": True, "dtype": "f32", "scaling": "linear", "far": 20000},
        # One decoding step of 64 requests: rotated, quantized and appended, the
        # queries rotated beside.
        {"name": "append-rope-decode-64", "op": "append", "R": 64, "L": 4096, "new": 1, "page": 64, "Hq": 32, "Hkv": 8,
         "d": 128, "rot": 128, "interleaved": False, "scaling": "parts", "packed": True},
        # Chunks of prompts, ending and starting anywhere in a page.
        {"name": "append-rope-prompts", "op": "append", "R": 9, "L": 1000, "new": 4096, "page": 128, "Hq": 32, "Hkv": 8,
         "d": 128, "rot": 128, "interleaved": False, "scaling": "none", "packed": True},
        # A short sequence: one tile of queries, latency.
        {"name": "dropout-fwd-100", "op": "attend", "bwd": False, "B": 1, "Hq": 8, "Hkv": 2, "N": 100, "d": 64,
         "causal": True, "p": 0.1},
        # The 1024-token workload (d = 64, every key seen) and the benchmark's
        # (4096 tokens, d = 128, causal), each forward and backward.
        {"name": "dropout-fwd-1024", "op": "attend", "bwd": False, "B": 4, "Hq": 16, "Hkv": 16, "N": 1024, "d": 64,
         "causal": False, "p": 0.1},
        {"name": "dropout-fwd-4096", "op": "attend", "bwd": False, "B": 2, "Hq": 32, "Hkv": 32, "N": 4096, "d": 128,
         "causal": True, "p": 0.1},
        # A ragged length with shared key/value heads.
        {"name": "dropout-bwd-777", "op": "attend", "bwd": True, "B": 2, "Hq": 12, "Hkv": 4, "N": 777, "d": 128,
         "causal": True, "p": 0.25},
        {"name": "dropout-bwd-1024", "op": "attend", "bwd": True, "B": 4, "Hq": 16, "Hkv": 16, "N": 1024, "d": 64,
         "causal": False, "p": 0.1},
        {"name": "dropout-bwd-4096", "op": "attend", "bwd": True, "B": 2, "Hq": 32, "Hkv": 32, "N": 4096, "d": 128,
         "causal": True, "p": 0.1},
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "attend"))
    Hq, Hkv = rng.choice(HEADS)
    d = rng.choice((64, 128))
    rot = rng.choice((d, d, d // 2, 16 * rng.randrange(1, d // 16 + 1)))
    common = {"op": op, "Hq": Hq, "Hkv": Hkv, "d": d}
    if op == "rope":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        most = 2 * 4096 * 64 * 128 // ((Hq + Hkv) * d * (2 if dtype == "f32" else 1))  # the tokens of the largest listed
        B = rng.choice((1, 1, 2, 3, 5))
        layout = rng.choice(("tokens", "packed", "heads")) if B == 1 else rng.choice(("packed", "heads"))
        return {**common, "bwd": rng.random() < 0.5, "layout": layout, "B": B, "N": _loguniform(rng, 1, most // B),
                "rot": rot, "interleaved": rng.random() < 0.5, "dtype": dtype, "scaling": rng.choice(SCALING),
                "far": rng.choice((0, _loguniform(rng, 1, 1000000)))}
    if op == "append":
        R = _loguniform(rng, 1, 600)
        new = 1 if rng.random() < 0.4 else _loguniform(rng, 1, max(1, 25000000 // (R * max(Hkv, Hq // 4) * d)))
        return {**common, "R": R, "L": _loguniform(rng, 1, max(2, 300000 // R)), "new": new, "page": rng.choice(PAGES),
                "rot": rot, "interleaved": rng.random() < 0.5, "scaling": rng.choice(SCALING),
                "packed": rng.random() < 0.5}
    B = rng.choice((1, 1, 2, 4))
    most = int(math.sqrt(64 * 4096 * 4096 / (2 * B * Hq)))  # the products of the largest listed, which is causal
    return {**common, "bwd": rng.random() < 0.5, "B": B, "N": _loguniform(rng, 1, min(4096, most)),
            "causal": rng.random() < 0.6, "p": rng.choice((0.05, 0.1, 0.2, 0.5, round(rng.uniform(0.01, 0.9), 3)))}


def _lengths(case):
    """(cached, new) of each request of an append, by the case alone."""
    R, L, new = case["R"], case["L"], case["new"]
    parts = [((r * 0.6180339887498949) % 1.0, (r * 0.7548776662466927) % 1.0) for r in range(R)]
    return [(round(L * (1 - 0.75 * u)), 1 if new == 1 else max(1, round(new * (1 - 0.9 * v)))) for u, v in parts]


def _pages_of(n, page):
    return -(-n // page)


def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        rows = case["B"] * case["N"] * (Hq + Hkv)
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * rows * d * size + 4 * case["B"] * case["N"] + 4 * case["rot"], "flops": 3 * rows * case["rot"]}
    if case["op"] == "append":
        T = sum(n for _, n in _lengths(case))
        return {"bytes": (4 * Hq + 6 * Hkv) * T * d + 12 * T + 4 * case["rot"],
                "flops": 3 * T * (Hq + Hkv) * case["rot"] + 4 * T * Hkv * d}
    B, N = case["B"], case["N"]
    kept = N * (N + 1) // 2 if case["causal"] else N * N
    if case["bwd"]:
        return {"bytes": 2 * B * N * d * (4 * Hq + 4 * Hkv) + 4 * B * Hq * N, "flops": 10 * B * Hq * kept * d}
    return {"bytes": 2 * B * N * d * (2 * Hq + 2 * Hkv) + 4 * B * Hq * N, "flops": 4 * B * Hq * kept * d}


# ------------------------------------------------------------------ inputs
def _frequencies(rot, scaling):
    """(turns a position of each pair, times 2^64, as int64; amplitude): base 10000, and for contexts
    eight times the original 4096 tokens either divided throughout or by parts: pairs that turn less than
    once over the original length divided, those that turn more than 32 times left, a ramp between."""
    f = [10000.0 ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)]
    amplitude = 1.0
    if scaling == "linear":
        f = [x / 8 for x in f]
    elif scaling == "parts":
        left = [min(1.0, max(0.0, (4096 * x - 1) / 31)) for x in f]
        f = [x / 8 * (1 - g) + x * g for x, g in zip(f, left)]
        amplitude = 0.1 * math.log(8.0) + 1
    return torch.tensor([round(x * 2.0 ** 64) for x in f], dtype=torch.int64, device="cuda"), amplitude


def _power_scale(amax):
    """The smallest power of two 2^k (k >= -126) with amax <= 448 * 2^k, in fp32."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax > 0, k, torch.full_like(k, -126)).clamp(min=-126)
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _values(shape, gen):
    """Keys or values as a projection gives them: normal, a few channels larger."""
    x = torch.randn(shape, generator=gen, device="cuda")
    gain = torch.exp2(torch.randn(shape[-1], generator=gen, device="cuda").clamp(-2, 2))
    return x * gain


def _filled_pages(num_pages, Hkv, page, d, gen):
    codes = torch.empty(num_pages, Hkv, page, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(num_pages, Hkv, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * d))
    for i in range(0, num_pages, step):
        x = _values((min(step, num_pages - i), Hkv, page, d), gen)
        s = _power_scale(x.abs().amax((2, 3)))
        codes[i:i + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[i:i + step] = s
    return codes, scales


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"rope": _prepare_rope, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](case, seed, gen)


def _prepare_rope(case, seed, gen):
    B, N, Hq, Hkv, d = (case[k] for k in ("B", "N", "Hq", "Hkv", "d"))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    freqs, amplitude = _frequencies(case["rot"], case["scaling"])
    s = {"op": "rope", "bwd": case["bwd"], "freqs": freqs, "interleaved": case["interleaved"], "amplitude": amplitude,
         "positions": None, "out": (None, None)}
    if case["far"]:
        if case["layout"] == "tokens":  # a token of each of N requests
            s["positions"] = torch.randint(0, case["far"], (N,), generator=gen, device="cuda").int()
        else:  # sequences that go on where others stopped
            first = torch.randint(0, case["far"], (B, 1), generator=gen, device="cuda")
            s["positions"] = (first + torch.arange(N, device="cuda")).int()
    if case["layout"] == "tokens":
        x = _values((N, Hq + 2 * Hkv, d), gen).to(dt)
        s.update(Q=x[:, :Hq], K=x[:, Hq:Hq + Hkv])
    elif case["layout"] == "packed" and not case["bwd"]:
        x = _values((B, N, Hq + 2 * Hkv, d), gen).to(dt).transpose(1, 2)
        s.update(Q=x[:, :Hq], K=x[:, Hq:Hq + Hkv])
    else:
        s.update(Q=_values((B, Hq, N, d), gen).to(dt), K=_values((B, Hkv, N, d), gen).to(dt))
        if case["layout"] == "packed":  # into the projection's gradient
            g = torch.zeros(B, N, Hq + 2 * Hkv, d, dtype=dt, device="cuda").transpose(1, 2)
            s["out"] = g[:, :Hq], g[:, Hq:Hq + Hkv]
    return s


def _prepare_append(case, seed, gen):
    page, R, Hq, Hkv, d = (case[k] for k in ("page", "R", "Hq", "Hkv", "d"))
    ln = _lengths(case)
    random.Random(seed).shuffle(ln)
    T = sum(n for _, n in ln)
    full = [_pages_of(c + n, page) for c, n in ln]
    num_pages = sum(full) + 3
    ids = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(R, max(full), dtype=torch.int32, device="cuda")
    table[torch.arange(max(full), device="cuda")[None, :] < _i32(full)[:, None]] = ids[:sum(full)]
    k_pages, k_scale = _filled_pages(num_pages, Hkv, page, d, gen)
    v_pages, v_scale = _filled_pages(num_pages, Hkv, page, d, gen)
    freqs, amplitude = _frequencies(case["rot"], case["scaling"])
    s = {"op": "append", "freqs": freqs, "interleaved": case["interleaved"], "amplitude": amplitude,
         "pages": (k_pages, k_scale, v_pages, v_scale)}
    if case["packed"]:
        x = _values((T, Hq + 2 * Hkv, d), gen).to(torch.bfloat16)
        s.update(Q=x[:, :Hq], K=x[:, Hq:Hq + Hkv], V=x[:, Hq + Hkv:])
    else:
        s.update({k: _values((T, h, d), gen).to(torch.bfloat16) for k, h in (("Q", Hq), ("K", Hkv), ("V", Hkv))})
    added = _i32([n for _, n in ln]).long()
    req = torch.repeat_interleave(torch.arange(R, device="cuda"), added)
    pos = torch.arange(T, device="cuda") - (torch.cumsum(added, 0) - added)[req] + _i32([c for c, _ in ln]).long()[req]
    s["positions"] = pos.int()
    s["slots"] = table[req, pos // page].long() * page + pos % page
    return s


def _prepare_attend(case, seed, gen):
    B, N, Hq, Hkv, d = (case[k] for k in ("B", "N", "Hq", "Hkv", "d"))
    s = {"op": "attend", "bwd": case["bwd"], "causal": case["causal"], "p": case["p"], "scale": 1.0 / math.sqrt(d)}
    for k, h in (("Q", Hq), ("K", Hkv), ("V", Hkv)):
        s[k] = torch.randn(B, h, N, d, generator=gen, device="cuda").to(torch.bfloat16)
    s["rng"] = torch.randint(0, 2 ** 62, (2,), generator=gen, device="cuda")  # seed; offset (its low 32 bits count)
    if case["bwd"]:
        s["dO"] = torch.randn(B, Hq, N, d, generator=gen, device="cuda").to(torch.bfloat16)
        s["O"], s["LSE"] = _plain_forward(s)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"rope": _run_rope, "append": _run_append, "attend": _run_attend}[s["op"]](s)


def _turned(X, freqs, positions, interleaved, amplitude, sign):
    """X [..., d] in 64 bits, rotated; positions broadcast against X's leading dimensions."""
    rot = 2 * freqs.numel()
    angle = torch.remainder(positions.double()[..., None] * (freqs.double() * 2.0 ** -64), 1.0) * (2 * math.pi)
    c, s = amplitude * torch.cos(angle), sign * amplitude * torch.sin(angle)
    x = X.double()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, z = a * c - b * s, b * c + a * s
    turned = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _run_rope(s):
    Q, K, positions, out = s["Q"], s["K"], s["positions"], s["out"]
    if own:
        f = _pkg().attn_rope_bwd if s["bwd"] else _pkg().attn_rope
        return f(Q, K, s["freqs"], positions, s["interleaved"], s["amplitude"], out[0], out[1])
    tokens = Q.dim() == 3
    if positions is None:
        positions = torch.arange(Q.shape[0] if tokens else Q.shape[2], device=Q.device)
    if tokens:
        positions = positions[:, None]
    elif positions.dim() == 2:
        positions = positions[:, None]
    sign = -1.0 if s["bwd"] else 1.0
    got = [_turned(X, s["freqs"], positions, s["interleaved"], s["amplitude"], sign).to(X.dtype) for X in (Q, K)]
    return tuple(g if o is None else o.copy_(g) for g, o in zip(got, out))


def _append_one(x, slots, pages, scales):
    num_pages, Hkv, page, d = pages.shape
    pg, off = slots // page, slots % page
    amax = torch.zeros_like(scales).index_reduce_(0, pg, x.abs().amax(2), "amax")
    lowest = torch.full((num_pages,), page, device=slots.device).scatter_reduce_(0, pg, off, "amin")
    touched = torch.unique(pg)
    old = torch.where(lowest[touched, None] > 0, scales[touched], 0.0)
    new = torch.maximum(old, _power_scale(amax[touched]))
    # Codes that were there before the first new token, at the new scale.
    have = torch.arange(page, device=slots.device)[None, :] < lowest[touched, None]
    ratio = torch.where(old > 0, old / new, 1.0)
    was = pages[touched]
    again = (was.view(torch.float8_e4m3fn).float() * ratio[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    pages[touched] = torch.where(have[:, None, :, None], again, was)
    scales[touched] = new
    pages[pg, :, off] = (x / scales[pg][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _run_append(s):
    pages = s["pages"]
    if own:
        q = _pkg().attn_kv_append_rope_fp8(s["Q"], s["K"], s["V"], s["positions"], s["slots"], s["freqs"], *pages,
                                           s["interleaved"], s["amplitude"])
    else:
        q, k = (_turned(X, s["freqs"], s["positions"][:, None], s["interleaved"], s["amplitude"], 1.0)
                for X in (s["Q"], s["K"]))
        q = q.to(torch.bfloat16)
        _append_one(k.float(), s["slots"], pages[0], pages[1])
        _append_one(s["V"].float(), s["slots"], pages[2], pages[3])
    # The codes as the e4m3 values that they are.
    return q, pages[0].view(torch.float8_e4m3fn), pages[1], pages[2].view(torch.float8_e4m3fn), pages[3]


def _philox(c, k):
    """Four words of Philox4x32 with seven rounds; all numbers in int64, whose products keep their low 64 bits."""
    for _ in range(7):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = ((q >> 32) & M32) ^ c[1] ^ k[0], q & M32, ((p >> 32) & M32) ^ c[3] ^ k[1], p & M32
        k = (k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32
    return c


def _kept(rng, p, B, Hq, N):
    """bool [B, Hq, N, N]: which elements of the softmax stay."""
    groups = _pages_of(N, 32)
    dev = rng.device
    half = torch.arange(2 * groups, device=dev)
    zero = torch.zeros(B * Hq, N, 2 * groups, dtype=torch.int64, device=dev)
    words = _philox((zero + torch.arange(N, device=dev)[:, None], zero + half,
                     zero + torch.arange(B * Hq, device=dev)[:, None, None], zero + (rng[1] & M32)),
                    (rng[0] & M32, (rng[0] >> 32) & M32))
    w = torch.stack(words, -1).reshape(B * Hq, N, groups, 8, 1)
    bit = torch.arange(32, device=dev)
    u = sum((((w[..., k, :] >> bit) & 1) << k).to(torch.uint8) for k in range(8))
    return (u.reshape(B, Hq, N, -1)[..., :N] >= _threshold(p))


def _threshold(p):
    return math.floor(256 * p + 0.5)


def _softmax(s):
    """(the softmax, its row maxima plus logarithms of sums), in 32 bits, and the shared heads of K and V repeated."""
    G = s["Q"].shape[1] // s["K"].shape[1]
    k, v = (s[n].float().repeat_interleave(G, 1) for n in "KV")
    x = torch.matmul(s["Q"].float(), k.transpose(2, 3)) * s["scale"]
    if s["causal"]:
        i = torch.arange(x.shape[2], device=x.device)
        x.masked_fill_(i[None, :] > i[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    return e / z, (m + torch.log(z))[..., 0], k, v


def _plain_forward(s):
    P, lse, _, v = _softmax(s)
    B, Hq, N, _ = s["Q"].shape
    P = torch.where(_kept(s["rng"], s["p"], B, Hq, N), P, 0.0)
    return (torch.matmul(P, v) / (1 - _threshold(s["p"]) / 256)).to(torch.bfloat16), lse


def _run_attend(s):
    if not s["bwd"]:
        if own:
            return _pkg().attn_fwd_dropout(s["Q"], s["K"], s["V"], s["p"], s["rng"], s["scale"], s["causal"])
        return _plain_forward(s)
    if own:
        return _pkg().attn_bwd_dropout(s["Q"], s["K"], s["V"], s["O"], s["dO"], s["LSE"], s["p"], s["rng"], s["scale"],
                                       s["causal"])
    B, Hq, N, d = s["Q"].shape
    Hkv = s["K"].shape[1]
    P, _, k, v = _softmax(s)
    keep = _kept(s["rng"], s["p"], B, Hq, N)
    mul = 1 / (1 - _threshold(s["p"]) / 256)
    g = s["dO"].float()
    dV = torch.matmul(torch.where(keep, P, 0.0).transpose(2, 3), g) * mul
    dP = torch.where(keep, torch.matmul(g, v.transpose(2, 3)) * mul, 0.0)
    dS = P * (dP - (g * s["O"].float()).sum(-1, keepdim=True)) * s["scale"]
    dQ, dK = torch.matmul(dS, k), torch.matmul(dS.transpose(2, 3), s["Q"].float())
    return (dQ.to(torch.bfloat16), *(t.reshape(B, Hkv, -1, N, d).sum(2).to(torch.bfloat16) for t in (dK, dV)))


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_turned(X, freqs, positions, interleaved, amplitude, sign):
    """X [rows, heads, d] with a position a row, as complex numbers times e^(i angle)."""
    rot = 2 * freqs.numel()
    # Whole products in units of 2^-64 turn: what passes 64 bits is whole turns.
    part = positions.long()[:, None] * freqs
    turn = (part >> 32).double() * 2.0 ** -32 + (part & M32).double() * 2.0 ** -64
    z = amplitude * torch.exp(torch.complex(torch.zeros_like(turn), sign * 2 * math.pi * turn))[:, None]
    x = X.double()
    pair = (x[..., :rot].unflatten(-1, (rot // 2, 2)) if interleaved
            else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2))
    w = torch.view_as_real(torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * z)
    w = w.flatten(-2) if interleaved else w.transpose(-1, -2).flatten(-2)
    return torch.cat((w, x[..., rot:]), -1)


def _nearest_e4m3(x):
    """The e4m3 value nearest to each element (ties to the even one), |x| <= 448."""
    a = x.abs()
    _, e = torch.frexp(a)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def _e4m3_values(codes):
    c = codes.long()
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.double() - 7), f * 2.0 ** -9)
    return torch.where(c >= 128, -v, v)


def _exact_append(X, slots, codes, scales):
    page = codes.shape[2]
    vals, sc = _e4m3_values(codes), scales.double()
    groups = {}
    for t, s in enumerate(slots.tolist()):
        groups.setdefault(s // page, []).append((t, s % page))
    for p, toks in groups.items():
        t0, off = toks[0]
        x = X[t0:t0 + len(toks)].double().transpose(0, 1)  # [Hkv, tokens, d]
        a = x.abs().amax((1, 2))
        k = torch.ceil(torch.log2(torch.where(a > 0, a, 1.0) / 448))
        k = torch.where(448 * torch.exp2(k - 1) >= a, k - 1, k)  # the logarithm may be just above a whole number
        k = torch.where(448 * torch.exp2(k) < a, k + 1, k).clamp(min=-126)
        want = torch.where(a > 0, torch.exp2(k), 2.0 ** -126)
        new = torch.maximum(want, sc[p]) if off > 0 else want
        if off > 0:
            vals[p, :, :off] = _nearest_e4m3(vals[p, :, :off] * (sc[p] / new)[:, None, None])
        vals[p, :, off:off + len(toks)] = _nearest_e4m3(x / new[:, None, None])
        sc[p] = new
    return vals, sc


def _exact_product(a, b):
    """(high, low) 32 bits of the product of two 32-bit numbers, by halves of 16 bits."""
    al, ah, bl, bh = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
    mid = (al * bl >> 16) + (al * bh & 0xFFFF) + (ah * bl & 0xFFFF)
    return ah * bh + (al * bh >> 16) + (ah * bl >> 16) + (mid >> 16), (mid & 0xFFFF) << 16 | (al * bl & 0xFFFF)


def _exact_numbers(rng, head, N):
    """u of the elements of one head: int64 [N, N]."""
    seed, offset = (int(v) for v in rng.tolist())
    i, j = torch.arange(N, device="cuda")[:, None], torch.arange(_pages_of(N, 32) * 2, device="cuda")[None, :]
    c = [i.expand(N, j.numel()), j.expand(N, j.numel()), torch.full((N, j.numel()), head, device="cuda"),
         torch.full((N, j.numel()), offset % 2 ** 32, device="cuda")]
    for r in range(7):
        k0, k1 = (seed + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        h0, l0 = _exact_product(c[0], 0xD2511F53)
        h1, l1 = _exact_product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
    w = torch.stack([x.unflatten(1, (-1, 2)) for x in c], -1).flatten(2)  # [N, groups, 8]
    bits = w[:, :, None, :] >> torch.arange(32, device="cuda")[:, None] & 1
    return (bits * 2 ** torch.arange(8, device="cuda")).sum(-1).flatten(1)[:, :N]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        sign = -1.0 if case["bwd"] else 1.0
        out = []
        for X in (s["Q"], s["K"]):
            rows = X if X.dim() == 3 else X.transpose(1, 2).reshape(-1, X.shape[1], X.shape[3])
            n = case["N"]
            pos = torch.arange(n, device="cuda") if s["positions"] is None else s["positions"]
            pos = pos.reshape(-1).repeat(rows.shape[0] // pos.numel())
            y = _exact_turned(rows, s["freqs"], pos, s["interleaved"], s["amplitude"], sign)
            out.append(y if X.dim() == 3 else y.reshape(X.shape[0], n, X.shape[1], -1).transpose(1, 2))
        return tuple(out)
    if case["op"] == "append":
        q, k = (_exact_turned(X, s["freqs"], s["positions"], s["interleaved"], s["amplitude"], 1.0)
                for X in (s["Q"], s["K"]))
        pages = s["pages"]
        return (q, *_exact_append(k, s["slots"], pages[0], pages[1]), *_exact_append(s["V"], s["slots"], pages[2], pages[3]))
    B, Hq, N, d = s["Q"].shape
    Hkv = s["K"].shape[1]
    T = _threshold(case["p"])
    late = torch.arange(N, device="cuda")[None, :] > torch.arange(N, device="cuda")[:, None]
    made = {k: torch.zeros(B, h, N, d, dtype=torch.float64, device="cuda")
            for k, h in (("O", Hq), ("dQ", Hq), ("dK", Hkv), ("dV", Hkv))}
    lse = torch.zeros(B, Hq, N, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(Hq):
            g = h * Hkv // Hq
            q, k, v = s["Q"][b, h].double(), s["K"][b, g].double(), s["V"][b, g].double()
            x = q @ k.T * s["scale"]
            if case["causal"]:
                x = x.masked_fill(late, -math.inf)
            factor = (_exact_numbers(s["rng"], b * Hq + h, N) >= T) * (256 / (256 - T))
            if not case["bwd"]:
                lse[b, h] = torch.logsumexp(x, -1)
                made["O"][b, h] = (torch.softmax(x, -1) * factor) @ v
                continue
            P, dO = torch.softmax(x, -1), s["dO"][b, h].double()
            D = (dO * s["O"][b, h].double()).sum(-1, keepdim=True)  # (O is an input: as it was stored)
            dS = P * ((dO @ v.T) * factor - D)
            made["dQ"][b, h] = s["scale"] * dS @ k
            made["dK"][b, g] += s["scale"] * dS.T @ q
            made["dV"][b, g] += (P * factor).T @ dO
    return (made["dQ"], made["dK"], made["dV"]) if case["bwd"] else (made["O"], lse)
