"""The paged cache's calls as a server strings them together: step after step
with nothing between the calls, first calls of a process inside a capture,
and caches whose offsets pass 32 bits, compared bit for bit with the same calls
made one at a time; and small decoding steps, whose tables' width decides how
the work is divided, against the plain 64-bit implementation."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import exact_attention_95_gb300 as pkg

import paged
from test_paged_cache import _cache, _check_attention, dev, dev_bf16

pytestmark = pytest.mark.gpu


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def _empty_cache(num_pages, Hkv, page, d, make=torch.zeros):
    return [x for _ in range(2) for x in (make(num_pages, Hkv, page, d, dtype=torch.uint8, device="cuda"),
                                          torch.ones(num_pages, Hkv, device="cuda"))]


@pytest.mark.parametrize("R,chunk", [(3, 0), (40, 0), (3, 90)])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_steps_with_nothing_between_the_calls(R, chunk, d, page):
    """Each append changes codes and scales that the attention before it reads
    (growing elements raise the scales), and each attention reuses the workspace
    of the one before.  chunk: every third step, request 0 takes that many tokens."""
    Hq, Hkv, steps, first = 8, 2, 24, 70
    g = torch.Generator(device="cuda").manual_seed(5)
    news = [[chunk if chunk and r == 0 and s % 3 == 2 else 1 for r in range(R)] for s in range(steps)]
    total = [first + sum(n[r] for n in news) for r in range(R)]
    width = max(-(-n // page) for n in total)
    num_pages = R * width
    table = torch.randperm(num_pages, generator=g, device="cuda").int().reshape(R, width).contiguous()
    steps_in = []
    lens = [0] * R
    for n in [[first] * R] + news:
        T = sum(n)
        grow = 2.0 ** (len(steps_in) / 4)
        slots = []
        for r in range(R):
            pos = lens[r] + torch.arange(n[r], device="cuda")
            slots.append(table[r].long()[pos // page] * page + pos % page)
        lens = [a + b for a, b in zip(lens, n)]
        steps_in.append((_randn(g, T, Hq, d), grow * _randn(g, T, Hkv, d), grow * _randn(g, T, Hkv, d),
                         torch.cat(slots), torch.tensor([0] + n, device="cuda").cumsum(0).int(),
                         torch.tensor(lens, dtype=torch.int32, device="cuda")))
    ws = torch.empty(max(pkg.attn_fwd_paged_workspace_size(R, x[0].shape[0], Hq, Hkv, d) for x in steps_in),
                     dtype=torch.uint8, device="cuda")

    def run(wait):
        cache = _empty_cache(num_pages, Hkv, page, d)
        outs = [(torch.empty_like(x[0]), torch.empty(x[0].shape[:2], device="cuda")) for x in steps_in]
        torch.cuda.synchronize()
        for (q, k, v, slots, cu, kv), (O, L) in zip(steps_in, outs):
            pkg.attn_kv_append_fp8(k, v, slots, *cache)
            if wait:
                torch.cuda.synchronize()
            pkg.attn_fwd_paged_fp8(q, *cache, table, cu, kv, causal=True, O=O, LSE=L, workspace=ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert pkg.attn_last_device_status() == pkg.ATTN_OK
        return [x for o in outs for x in o] + cache

    want = run(True)
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("chunk", [1, 40])
def test_offsets_past_32_bits(chunk):
    """The same tokens in pages at the end of 5 GB of keys and 5 GB of values and in a small cache."""
    page, Hkv, d, Hq = 128, 8, 128, 16
    num_pages, used, lens = 40000, 8, [500, 130]
    assert num_pages * Hkv * page * d > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(6)
    T = sum(lens)
    k, v = _randn(g, T, Hkv, d), _randn(g, T, Hkv, d)
    q = _randn(g, 2 * chunk, Hq, d)
    cu = torch.tensor([0, chunk, 2 * chunk], dtype=torch.int32, device="cuda")
    added = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = []
    for n in (used, num_pages):
        cache = _empty_cache(n, Hkv, page, d, torch.empty)
        free = torch.arange(n - used, n, dtype=torch.int32, device="cuda")
        table = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
        kv, _, slots, _, _ = pkg.attn_kv_tables(torch.zeros_like(added), added, free, table, page, T)
        pkg.attn_kv_append_fp8(k, v, slots, *cache)
        got.append(pkg.attn_fwd_paged_fp8(q, *cache, table, cu, kv, causal=True))
        torch.cuda.synchronize()
        assert pkg.attn_last_device_status() == pkg.ATTN_OK
        assert int(slots.max()) == (n - used + 5) * page + 130 - page - 1
        got[-1] += tuple(x[n - used:n - used + 6].clone() for x in cache)
        del cache
    rows = torch.arange(page, device="cuda")
    for a, b in zip(got[0][:2], got[1][:2]):
        assert torch.equal(a, b)
    for i in (2, 3, 4, 5):
        a, b = got[0][i], got[1][i]
        if a.dim() == 4:  # codes of the places that hold tokens
            held = torch.stack([rows < (x - y * page) for x, y in [(500, 0), (500, 1), (500, 2), (500, 3), (130, 0),
                                                                   (130, 1)]])[:, None, :, None]
            a, b = (x * held for x in (a, b))
        assert torch.equal(a, b)


def test_threads_with_a_stream_each():
    """Calls of four threads at once (the binding lets Python's lock go) against the same calls in turn."""
    g = torch.Generator(device="cuda").manual_seed(9)
    Hq, Hkv, d, page = 16, 4, 64, 16
    work = []
    for i, (R, new) in enumerate([(2, 1), (5, 3), (40, 1), (1, 60)]):
        T = R * new
        cache = _empty_cache(400, Hkv, page, d)
        free = torch.randperm(400, generator=g, device="cuda").int()
        added = torch.full((R,), new, dtype=torch.int32, device="cuda")
        work.append((_randn(g, T, Hq, d), _randn(g, T, Hkv, d), _randn(g, T, Hkv, d), cache, free, added, R, T))

    def steps(w):
        q, k, v, cache, free, added, R, T = w
        table = torch.zeros(R, 20, dtype=torch.int32, device="cuda")
        cached = torch.zeros_like(added)
        out = []
        for s in range(5):  # (one request takes four pages a step, the others none after the first)
            kv, cu, slots, _, _ = pkg.attn_kv_tables(cached, added, free[8 * s:], table, page, T)
            pkg.attn_kv_append_fp8(k, v, slots, *cache)
            out += pkg.attn_fwd_paged_fp8(q, *cache, table, cu, kv, causal=True)
            cached = kv
        return out

    def reset(w):
        for x in w[3]:
            x.fill_(1)

    for w in work:
        reset(w)
    want = [steps(w) for w in work]
    torch.cuda.synchronize()
    for w in work:
        reset(w)
    torch.cuda.synchronize()
    got, streams = [None] * 4, [torch.cuda.Stream() for _ in work]

    def run(i):
        with torch.cuda.stream(streams[i]):
            got[i] = steps(work[i])
            streams[i].synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK
    for a, b in zip(got, want):
        assert a is not None and all(torch.equal(x, y) for x, y in zip(a, b))


FIRST = """
import torch
import exact_attention_95_gb300 as pkg
dev = "cuda"
R, Hq, Hkv, d, page = 3, 8, 2, %d, 32
g = torch.Generator(device=dev).manual_seed(1)
new = %d
T = R * new
q, k, v = (torch.randn(T, h, d, generator=g, device=dev).bfloat16() for h in (Hq, Hkv, Hkv))
cache = [x for _ in range(2) for x in (torch.zeros(40, Hkv, page, d, dtype=torch.uint8, device=dev),
                                       torch.ones(40, Hkv, device=dev))]
cached = torch.zeros(R, dtype=torch.int32, device=dev)
added = torch.full((R,), new, dtype=torch.int32, device=dev)
free = torch.arange(40, dtype=torch.int32, device=dev)
table = torch.zeros(R, 8, dtype=torch.int32, device=dev)
def step():
    kv, cu, slots, _, _ = pkg.attn_kv_tables(cached, added, free, table, page, T)
    pkg.attn_kv_append_fp8(k, v, slots, *cache)
    return pkg.attn_fwd_paged_fp8(q, *cache, table, cu, kv, causal=True)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in out]
want = step()
torch.cuda.synchronize()
assert pkg.attn_last_device_status() == pkg.ATTN_OK
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert float(got[0].float().abs().max()) > 0
print("captured first")
"""


@pytest.mark.parametrize("d,new", [(64, 1), (128, 50)])
def test_the_first_calls_of_a_process_inside_a_capture(d, new):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % (d, new)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


STEPS = [
    # lens, new tokens, Hq, Hkv, d, page
    ([1], [1], 1, 1, 64, 16),
    ([700, 20, 0, 351], [1, 1, 1, 1], 32, 8, 128, 16),
    ([5000], [1], 8, 1, 128, 128),              # 40 units of one item
    ([1023, 1024, 1025, 127, 128, 129], [1] * 6, 16, 8, 64, 32),
    ([300, 40, 0, 7, 90], [3, 0, 0, 1, 1], 8, 1, 64, 16),   # idle requests; several tokens and tiles of one
    ([2, 40, 9, 500], [4, 0, 0, 0], 7, 1, 128, 32),  # more queries than keys: the first rows see none
    ([100 * i for i in range(12)], [1] * 12, 32, 8, 128, 64),
    ([33] * 60, [0] * 57 + [1] * 3, 12, 2, 64, 16),  # more than 32 requests
]


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "R%d_Hq%d_Hkv%d_d%d_p%d" % (len(c[0]), *c[2:]))
@pytest.mark.parametrize("keys", [0, 10000])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_small_steps_with_narrow_and_wide_tables(case, keys, out):
    lens, news, Hq, Hkv, d, page = case
    rng = np.random.default_rng(51)
    kc, ks, vc, vs, table = _cache(rng, lens, page, Hkv, d, width_extra=1 + keys // page)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    T = int(cu[-1])
    assert T <= len(lens)
    q = paged.bf16_bits(rng.standard_normal((T, Hq, d)).astype(np.float32))
    g = [dev(a) for a in (kc, ks, vc, vs, table, cu, np.asarray(lens, np.int32))]
    O, L = pkg.attn_fwd_paged_fp8(dev_bf16(q), *g, None, True, out)
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK
    Or, Lr, A, B = paged.attention(paged.bf16_values(q), kc, ks, vc, vs, table, cu, lens,
                                   float(np.float32(1 / np.sqrt(d))), True)
    tol_o, tol_l = paged.bounds(Or, Lr, A, B, d, out == torch.bfloat16)
    none = np.isneginf(Lr)
    Og, Lg = O.double().cpu().numpy(), L.double().cpu().numpy()
    assert np.array_equal(np.isneginf(Lg), none) and (Og[none] == 0.0).all()
    assert (np.abs(Og - Or) <= tol_o).all()
    assert (np.abs(np.where(none, 0.0, Lg) - np.where(none, 0.0, Lr)) <= tol_l).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_value_in_a_small_step_with_narrow_and_wide_tables(d):
    """The NaN lies at the last key, which the last of a request's three tokens sees alone."""
    rng = np.random.default_rng(52)
    lens, Hq, Hkv, page = [300, 40, 60], 2, 1, 16
    cu = np.array([0, 3, 3, 3], np.int32)
    q = dev_bf16(paged.bf16_bits(rng.standard_normal((3, Hq, d)).astype(np.float32)))
    for extra in (1, 700):
        kc, ks, vc, vs, table = _cache(np.random.default_rng(53), lens, page, Hkv, d, width_extra=extra)
        vc[table[0, 299 // page], 0, 299 % page, 5] = 0x7F
        g = [dev(a) for a in (kc, ks, vc, vs, table, cu, np.asarray(lens, np.int32))]
        O, L = pkg.attn_fwd_paged_fp8(q, *g, None, True, torch.float32)
        torch.cuda.synchronize()
        assert pkg.attn_last_device_status() == pkg.ATTN_OK
        want = np.zeros((3, Hq, d), bool)
        want[2, :, 5] = True
        assert np.array_equal(torch.isnan(O).cpu().numpy(), want) and torch.isfinite(L).all()


@pytest.mark.parametrize("lens,news,Hq,Hkv,d,page,pad", [
    ([500], [3], 8, 2, 128, 32, 60),        # one request of a few rows among many places
    ([500], [0], 8, 2, 64, 32, 60),         # and of none
    ([3000, 2900], [12, 11], 16, 1, 128, 32, 0),  # two tall items in two dozen parts each
    ([3000], [12], 16, 1, 64, 128, 5),
    ([40, 9000], [2, 70], 8, 1, 64, 16, 0),
])
def test_few_tall_items(lens, news, Hq, Hkv, d, page, pad):
    for out in (torch.bfloat16, torch.float32):
        _check_attention(np.random.default_rng(61), lens, news, Hq, Hkv, d, page, True, out, pad=pad)
