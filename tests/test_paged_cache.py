"""The paged 8-bit key/value cache against its plain 64-bit implementation:
tables of a step (whole numbers: equal), the quantizing append (codes and
scales: equal), attention over the pages (within a bound derived from the
arithmetic, tests/paged.py), and the three together as a server runs them."""

import numpy as np
import pytest
import torch

import exact_attention_95_gb300 as pkg

import paged

gpu = pytest.mark.gpu
I32 = np.int32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def ok():
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK


# ------------------------------------------------------------------ plain implementation
def test_plain_power_scale_and_append_on_known_values():
    assert paged.power_scale(448.0) == 1.0 and paged.power_scale(448.1) == 2.0
    assert paged.power_scale(0.0) == 2.0 ** -126 and paged.power_scale(1.75) == 2.0 ** -8
    codes = np.zeros((2, 1, 16, 64), np.uint8)
    scales = np.ones((2, 1))
    x = np.zeros((2, 1, 64))
    x[0, 0, 0], x[1, 0, 1] = 448.0, 896.0
    c, s = paged.append(x, [15, 16], codes, scales)
    assert s[0, 0] == 1.0 and s[1, 0] == 2.0
    assert c[0, 0, 15, 0] == 0x7E and c[1, 0, 0, 1] == 0x7E
    # A later, larger token raises the page's scale and halves the codes before it.
    y = np.zeros((1, 1, 64))
    y[0, 0, 2] = 1792.0
    c2, s2 = paged.append(y, [17], c, s)
    assert s2[1, 0] == 4.0 and c2[1, 0, 0, 1] == 0x76 and c2[1, 0, 1, 2] == 0x7E


def test_plain_tables_on_a_hand_made_step():
    table = np.zeros((3, 3), I32)
    table[0, 0], table[2, :2] = 7, (4, 5)
    t, lens, cu, slots, pos, taken = paged.tables([15, 0, 30], [3, 0, 2], [9, 8], table, 16, 6)
    assert t[0, 1] == 9 and list(lens) == [18, 0, 32] and list(cu) == [0, 3, 3, 5]
    assert list(slots) == [7 * 16 + 15, 9 * 16, 9 * 16 + 1, 5 * 16 + 14, 5 * 16 + 15, -1]
    assert list(pos) == [15, 16, 17, 30, 31, -1] and list(taken) == [1, 0]


def test_plain_attention_equals_the_oracle_on_one_page():
    import oracle
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 0x70, (2, 1, 16, 64)).astype(np.uint8)
    scales = np.array([[0.01], [0.02]], np.float32)
    Q = rng.standard_normal((2, 2, 64))
    O, L, A, B = paged.attention(Q, codes, scales, codes[::-1], scales, np.array([[1, 0]]), [0, 2], [19], 0.2, True)
    k = paged.dequantize(codes, scales, [1, 0], 19)[None]
    v = paged.dequantize(codes[::-1], scales, [1, 0], 19)[None]
    Or, Lr = oracle.fwd(np.ascontiguousarray(Q.transpose(1, 0, 2)[None]), k, v, 0.2, True)
    assert np.abs(O - Or[0].transpose(1, 0, 2)).max() < 1e-12 and np.abs(L - Lr[0].T).max() < 1e-12
    assert (A >= np.abs(O) - 1e-12).all() and (B[0] > 0).all()


# ------------------------------------------------------------------ tables
def _step(rng, R, page, lo, hi, new, width=None, free=None):
    cached = rng.integers(lo, hi + 1, R).astype(I32)
    added = np.where(rng.random(R) < 0.2, 0, rng.integers(0, new + 1, R)).astype(I32)
    have = -(-cached // page)
    full = -(-(cached + added) // page)
    width = int(full.max()) + 1 if width is None else width
    ids = rng.permutation(int(have.sum() + (full - have).sum()) + 5).astype(I32)
    table = np.full((R, width), -7, I32)
    at = 0
    for r in range(R):
        n = min(int(have[r]), width)
        table[r, :n] = ids[at:at + n]
        at += n
    fr = ids[at:] if free is None else ids[at:at + free]
    return cached, added, table, np.ascontiguousarray(fr)


def _check_tables(cached, added, free, table, page, T):
    want = paged.tables(cached, added, free, table, page, T)
    tb = dev(table)
    got = pkg.attn_kv_tables(dev(cached), dev(added), dev(free), tb, page, T)
    ok()
    for name, w, g in zip(("block_table", "kv_lens", "cu_tokens", "slots", "positions", "taken"), want, (tb, *got)):
        assert np.array_equal(w, g.cpu().numpy().astype(np.int64)), name


@gpu
@pytest.mark.parametrize("R,page,lo,hi,new,pad", [
    (1, 64, 0, 0, 1, 0), (1, 16, 31, 31, 1, 3), (8, 64, 1, 4096, 1, 0), (257, 16, 0, 300, 40, 17),
    (1023, 32, 0, 100, 3, 0), (1025, 128, 0, 1000, 150, 5), (2500, 16, 0, 64, 33, 1), (3, 128, 0, 5, 9000, 100),
])
def test_tables_match_the_plain_form(R, page, lo, hi, new, pad):
    rng = np.random.default_rng(R + page)
    cached, added, table, free = _step(rng, R, page, lo, hi, new)
    _check_tables(cached, added, free, table, page, int(added.sum()) + pad)


@gpu
@pytest.mark.parametrize("kind", ["pages", "width", "places", "none"])
def test_tables_refuse_requests_that_do_not_fit(kind):
    rng = np.random.default_rng(11)
    for R in (40, 1500):
        cached, added, table, free = _step(rng, R, 16, 0, 100, 30, width=6 if kind == "width" else None)
        T = int(added.sum())
        if kind == "pages":
            free = free[:len(free) // 3]
        elif kind == "places":
            T = T * 2 // 3
        elif kind == "none":
            free = free[:0]
        _check_tables(cached, added, free, table, 16, T)


@gpu
def test_tables_clip_negative_and_huge_lengths():
    cached = np.array([-5, 10, 2 ** 31 - 1, 3, 0], I32)
    added = np.array([4, -1, 2 ** 31 - 1, 2, 2 ** 31 - 1], I32)
    table = np.arange(10, dtype=I32).reshape(5, 2)
    _check_tables(cached, added, np.arange(50, 60, dtype=I32), table, 16, 20)


@gpu
def test_tables_without_new_tokens_or_places():
    table = np.arange(6, dtype=I32).reshape(3, 2)
    _check_tables(np.array([3, 0, 20], I32), np.zeros(3, I32), np.zeros(0, I32), table, 16, 0)
    _check_tables(np.array([3, 0, 20], I32), np.zeros(3, I32), np.zeros(0, I32), table, 16, 4)


# ------------------------------------------------------------------ append
def _pages(rng, num_pages, Hkv, page, d, spread=3):
    codes = rng.integers(0, 256, (num_pages, Hkv, page, d)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x35
    scales = np.exp2(rng.integers(-9 - spread, -8 + spread, (num_pages, Hkv))).astype(np.float32)
    return codes, scales


def _tokens(rng, T, H, d, spread=4):
    x = rng.standard_normal((T, H, d)) * np.exp2(rng.integers(-spread, spread + 1, (T, H, 1)))
    return paged.bf16_bits(x.astype(np.float32))


def _check_append(kb, vb, slots, kc, ks, vc, vs, packed=0):
    wk = paged.append(paged.bf16_values(kb), slots, kc, ks)
    wv = paged.append(paged.bf16_values(vb), slots, vc, vs)
    T, H, d = kb.shape
    if packed:  # K and V as slices of [T, packed + 2 H, d]
        x = torch.zeros(T, packed + 2 * H, d, dtype=torch.bfloat16, device="cuda")
        x[:, packed:packed + H] = dev_bf16(kb)
        x[:, packed + H:] = dev_bf16(vb)
        K, V = x[:, packed:packed + H], x[:, packed + H:]
    else:
        K, V = dev_bf16(kb), dev_bf16(vb)
    g = [dev(a) for a in (kc, ks, vc, vs)]
    pkg.attn_kv_append_fp8(K, V, dev(np.asarray(slots, np.int64)), *g)
    ok()
    for name, w, x in zip(("k codes", "k scale", "v codes", "v scale"), (*wk, *wv), g):
        got = x.cpu().numpy()
        if got.dtype == np.uint8:  # -0 and +0 are the same value
            w, got = np.where(w == 0x80, 0, w), np.where(got == 0x80, 0, got)
        assert np.array_equal(w, got.astype(w.dtype)), name
    return g


@gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,packed", [(1, 0), (3, 5)])
def test_append_matches_the_plain_form(page, d, Hkv, packed):
    rng = np.random.default_rng(page + d + Hkv)
    num_pages = 40
    kc, ks = _pages(rng, num_pages, Hkv, page, d)
    vc, vs = _pages(rng, num_pages, Hkv, page, d)
    ids = rng.permutation(num_pages)
    slots, at = [], 0
    # Runs of one token to several pages, at any offset, with skipped tokens between them.
    for n in (1, 1, 2, 15, 16, 17, page - 1, page, page + 1, 2 * page + 5, 1):
        off = int(rng.integers(0, page))
        for i in range(n):
            if at >= num_pages:
                break
            slots.append(int(ids[at]) * page + off)
            off += 1
            if off == page:
                off, at = 0, at + 1
        if off:
            at += 1
        if n % 2:
            slots.append(-1 if n == 1 else num_pages * page)
    T = len(slots)
    _check_append(_tokens(rng, T, Hkv, d), _tokens(rng, T, Hkv, d), slots, kc, ks, vc, vs, packed)


@gpu
def test_append_of_many_tokens_and_of_none():
    rng = np.random.default_rng(5)
    page, Hkv, d = 64, 2, 128
    kc, ks = _pages(rng, 60, Hkv, page, d)
    vc, vs = _pages(rng, 60, Hkv, page, d)
    slots = (np.arange(3000) + 37).tolist()
    g = _check_append(_tokens(rng, 3000, Hkv, d), _tokens(rng, 3000, Hkv, d), slots, kc, ks, vc, vs)
    before = [x.clone() for x in g]
    e = torch.empty(0, Hkv, d, dtype=torch.bfloat16, device="cuda")
    pkg.attn_kv_append_fp8(e, e, torch.empty(0, dtype=torch.int64, device="cuda"), *g)
    pkg.attn_kv_append_fp8(dev_bf16(_tokens(rng, 3, Hkv, d)), dev_bf16(_tokens(rng, 3, Hkv, d)),
                           torch.full((3,), -1, dtype=torch.int64, device="cuda"), *g)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(g, before))


@gpu
def test_append_special_values():
    """Zeros, the smallest and largest bf16 numbers, values at the scale's borders, NaN and infinities."""
    page, d = 16, 64
    vals = [0.0, 2.0 ** -133, 2.0 ** -126, 448.0, 450.0, 1.75, 1.7578125, 3.3895314e38, 2.0 ** -120, -448.0]
    T = len(vals)
    x = np.zeros((T, 1, d), np.float32)
    for t, v in enumerate(vals):
        x[t, 0, :] = np.float32(v) * np.float32(0.5) ** (np.arange(d) % 24)
    bits = paged.bf16_bits(x)
    kc, ks = _pages(np.random.default_rng(1), T + 1, 1, page, d)
    slots = [t * page for t in range(T)]
    _check_append(bits, bits[::-1].copy(), slots, kc, ks, kc, ks)
    # Non-finite elements do not set the scale.
    b = bits[3:4].copy()
    b[0, 0, 3], b[0, 0, 5], b[0, 0, 7] = 0x7F80, 0xFF80, 0x7FC0
    ws = paged.append(paged.bf16_values(np.where((b & 0x7F80) == 0x7F80, 0, b)), [5], kc, ks)
    g = [dev(a) for a in (kc, ks, kc, ks)]
    pkg.attn_kv_append_fp8(dev_bf16(b), dev_bf16(b), dev(np.array([5], np.int64)), *g)
    ok()
    got = g[0].cpu().numpy()
    assert np.array_equal(g[1].cpu().numpy(), ws[1].astype(np.float32))
    assert got[0, 0, 5, 3] == 0x7E and got[0, 0, 5, 5] == 0xFE and got[0, 0, 5, 7] & 0x7F == 0x7F


@gpu
def test_append_token_by_token_equals_append_at_once():
    """With a power-of-two scale, growing a page token by token gives the codes of
    one call, but for those that became subnormal on the way."""
    rng = np.random.default_rng(8)
    page, Hkv, d, T = 32, 2, 64, 32
    k, v = (dev_bf16(_tokens(rng, T, Hkv, d, 1)) for _ in range(2))
    z = lambda: [torch.zeros(1, Hkv, page, d, dtype=torch.uint8, device="cuda"), torch.ones(1, Hkv, device="cuda"),
                 torch.zeros(1, Hkv, page, d, dtype=torch.uint8, device="cuda"), torch.ones(1, Hkv, device="cuda")]
    a, b = z(), z()
    slots = torch.arange(T, device="cuda")
    pkg.attn_kv_append_fp8(k, v, slots, *a)
    for t in range(T):
        pkg.attn_kv_append_fp8(k[t:t + 1], v[t:t + 1], slots[t:t + 1], *b)
    ok()
    assert torch.equal(a[1], b[1]) and torch.equal(a[3], b[3])
    for i in (0, 2):
        x, y = (c[i].view(torch.float8_e4m3fn).float() for c in (a, b))
        assert (x - y).abs().max().item() <= 2.0 ** -9  # one subnormal step
        normal = x.abs() >= 2.0 ** -5
        assert torch.equal(x[normal], y[normal])


# ------------------------------------------------------------------ attention
def _cache(rng, lens, page, Hkv, d, spread=2, width_extra=1):
    need = [-(-int(n) // page) for n in lens]
    num_pages = sum(need) + 3
    kc, ks = _pages(rng, num_pages, Hkv, page, d, spread)
    vc, vs = _pages(rng, num_pages, Hkv, page, d, spread)
    ids = rng.permutation(num_pages).astype(I32)
    table = np.full((len(lens), max(need + [1]) + width_extra), -1, I32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
        # Behind the last token a page holds anything, a NaN code too.
        tail = int(lens[r]) % page
        if tail:
            for c in (kc, vc):
                c[table[r, n - 1], :, tail:] = rng.choice([0x7F, 0xFF, 0x7E, 0x00], c[0, :, tail:].shape)
    return kc, ks, vc, vs, table


def _check_attention(rng, lens, news, Hq, Hkv, d, page, causal, out=torch.bfloat16, q_mul=1.0, pad=0, packed=0,
                     spread=2, uneven=False, **kw):
    kc, ks, vc, vs, table = _cache(rng, lens, page, Hkv, d, spread)
    if uneven:
        ks, vs = (s * rng.uniform(1, 2, s.shape).astype(np.float32) for s in (ks, vs))
    cu = np.concatenate([[0], np.cumsum(news)]).astype(I32)
    T = int(cu[-1]) + pad
    q = paged.bf16_bits((q_mul * rng.standard_normal((T, Hq, d))).astype(np.float32))
    Qd = dev_bf16(q)
    if packed:
        x = torch.zeros(T, Hq + packed, d, dtype=torch.bfloat16, device="cuda")
        x[:, :Hq] = Qd
        Qd = x[:, :Hq]
    O = torch.full((T, Hq, d), 7.0, dtype=out, device="cuda")
    L = torch.full((T, Hq), 7.0, device="cuda")
    scale = 1.0 / np.sqrt(d)
    g = [dev(a) for a in (kc, ks, vc, vs, table, cu, np.asarray(lens, I32))]
    pkg.attn_fwd_paged_fp8(Qd, *g, scale, causal, out, O, L, **kw)
    ok()
    Or, Lr, A, B = paged.attention(paged.bf16_values(q), kc, ks, vc, vs, table, cu, lens, float(np.float32(scale)),
                                   causal)
    tol_o, tol_l = paged.bounds(Or, Lr, A, B, d, out == torch.bfloat16)
    n = int(cu[-1])
    Og, Lg = O.double().cpu().numpy(), L.double().cpu().numpy()
    assert (Og[n:] == 7.0).all() and (Lg[n:] == 7.0).all(), "rows behind the last request were written"
    none = np.isneginf(Lr[:n])
    assert np.array_equal(np.isneginf(Lg[:n]), none)
    assert (Og[:n][none] == 0.0).all()
    err = np.abs(Og[:n] - Or[:n])
    assert (err <= tol_o[:n]).all(), f"O off by {np.nanmax(err / tol_o[:n]):.2f} of its bound"
    el = np.abs(np.where(none, 0.0, Lg[:n]) - np.where(none, 0.0, Lr[:n]))
    assert (el <= tol_l[:n]).all(), f"LSE off by {(el / tol_l[:n]).max():.2f} of its bound"


ATTENTION = [
    # lens, new tokens, Hq, Hkv, d, page, causal
    ([1], [1], 1, 1, 64, 16, True),
    ([5], [1], 4, 1, 128, 16, True),
    ([128], [1], 8, 2, 128, 128, False),
    ([129], [1], 8, 2, 64, 64, True),
    ([700, 1, 33, 0, 512], [1, 1, 1, 1, 1], 8, 2, 128, 16, True),
    ([700, 1, 33, 0, 512], [1, 0, 1, 2, 0], 8, 2, 128, 32, True),
    ([300, 40, 1000], [5, 40, 3], 6, 2, 64, 32, True),
    ([300, 40, 1000], [5, 60, 3], 6, 2, 128, 64, True),  # more queries than keys: the first rows see none
    ([300, 40, 1000], [5, 60, 3], 6, 2, 128, 64, False),
    ([257, 400], [17, 130], 32, 2, 128, 128, True),   # 16 heads a kv head
    ([90, 513], [2, 3], 40, 1, 64, 16, True),         # 40 heads a kv head: three row tiles a token
    ([4000], [1], 2, 2, 128, 128, True),
    ([9000], [3], 12, 4, 64, 16, False),
    # More than eight query rows of a kv head.
    ([600], [300], 4, 2, 128, 64, True),
    ([600, 0, 130], [300, 0, 130], 8, 2, 64, 16, True),
    ([1500, 20, 1], [7, 20, 1], 8, 1, 128, 32, True),   # wide and narrow requests in one call
    ([6000], [33], 8, 2, 128, 128, False),
    ([2100, 300], [1, 1], 32, 2, 128, 64, True),        # 16 heads a kv head, one token
    ([128, 129, 127], [128, 129, 127], 2, 2, 64, 128, True),
    ([200], [257], 1, 1, 128, 16, True),
    ([5000, 128, 300], [6, 5, 9], 32, 8, 128, 32, True),  # 17 to 128 rows
    ([5000, 128, 300], [30, 31, 32], 8, 2, 64, 64, True),
    ([700, 900], [100, 128], 1, 1, 128, 16, False),
    ([700, 900, 20], [128, 129, 100], 2, 2, 64, 16, True),
]


@gpu
@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "L%s_n%s_Hq%d_Hkv%d_d%d_p%d_c%d" % (
    "-".join(map(str, c[0])), "-".join(map(str, c[1])), *c[2:]))
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_attention_matches_the_plain_form(case, out):
    lens, news, Hq, Hkv, d, page, causal = case
    _check_attention(np.random.default_rng(sum(lens) + d), lens, news, Hq, Hkv, d, page, causal, out)


@gpu
@pytest.mark.parametrize("R", [70, 1100])
def test_attention_of_many_requests_some_idle(R):
    rng = np.random.default_rng(R)
    lens = rng.integers(0, 200, R)
    news = np.where(rng.random(R) < 0.4, 0, 1)
    _check_attention(rng, lens, news, 4, 2, 64, 16, True)


@gpu
@pytest.mark.parametrize("d,page", [(64, 32), (128, 16), (128, 128)])
def test_attention_of_many_units_a_worker(d, page):
    """Several times more 128-key units than the GPU has SMs times ring stages."""
    rng = np.random.default_rng(d + page)
    lens = rng.integers(1, 9000, 40)
    _check_attention(rng, lens, np.ones(40, int), 8, 4, d, page, True)


@gpu
def test_attention_padded_strided_and_with_a_callers_workspace():
    rng = np.random.default_rng(21)
    ws = torch.full((pkg.attn_fwd_paged_workspace_size(2, 8, 8, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    _check_attention(rng, [500, 77], [2, 1], 8, 2, 128, 64, True, pad=5, packed=4, workspace=ws)


@gpu
def test_attention_large_logits_and_uneven_page_scales():
    rng = np.random.default_rng(22)
    for news in ([1, 1], [1, 4], [40, 9]):
        _check_attention(rng, [2000, 300], news, 8, 2, 128, 16, True, torch.float32, q_mul=8.0)
        _check_attention(rng, [2000, 300], news, 8, 2, 128, 16, True, torch.float32, q_mul=0.05, spread=8)


@gpu
def test_attention_scales_that_are_no_powers_of_two():
    rng = np.random.default_rng(25)
    for news in ([1, 1], [40, 9]):
        _check_attention(rng, [700, 300], news, 8, 2, 64, 32, True, torch.float32, uneven=True)


@gpu
def test_attention_keeps_a_tail_behind_a_dominant_key():
    """One key 12 above the rest in the logit and a biased V: the tail's mass, tens of
    thousands of weights of 2^-17, has to reach O."""
    page, d, L = 128, 64, 40000
    n = -(-L // page)
    kc, vc = np.zeros((n, 1, page, d), np.uint8), np.full((n, 1, page, d), 0x38, np.uint8)  # V = 1
    kc[0, 0, 0, 0] = 0x38  # K_0 = (1, 0, ...)
    vc[0, 0, 0, :] = 0  # V_0 = 0
    one = np.ones((n, 1), np.float32)
    for T in (1, 20):  # a decoding step; many rows
        q = np.zeros((T, 1, d), np.float32)
        q[:, 0, 0] = 12.0
        g = [dev(a) for a in (kc, one, vc, one, np.arange(n, dtype=I32)[None], np.array([0, T], I32), np.array([L], I32))]
        O, Ls = pkg.attn_fwd_paged_fp8(dev_bf16(paged.bf16_bits(q)), *g, 1.0, False, torch.float32)
        ok()
        z = np.exp(12.0) + L - 1
        want = (L - 1) / z
        assert abs(O.cpu().numpy() - want).max() <= want * (2.0 ** -11 + 2.0 ** -15)
        assert abs(Ls.cpu().numpy() - np.log(z)).max() <= 1e-4


@gpu
def test_attention_reports_pages_out_of_range_and_lengths_past_the_table():
    rng = np.random.default_rng(23)
    kc, ks, vc, vs, table = _cache(rng, [100, 100], 16, 1, 64)
    good = table.copy()
    table[0, 2], table[1, 6] = 10 ** 9, -3
    q = _tokens(rng, 2, 2, 64, 0)
    args = [dev(a) for a in (kc, ks, vc, vs)]
    cu = dev(np.array([0, 1, 2], I32))
    O, L = pkg.attn_fwd_paged_fp8(dev_bf16(q), *args, dev(table), cu, dev(np.array([100, 100], I32)), 0.125, True,
                                  torch.float32)
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_ERR_DEVICE
    assert torch.isfinite(O).all() and torch.isfinite(L).all()
    # The keys of the bad page take no part: the same as without them.
    O2, L2 = pkg.attn_fwd_paged_fp8(dev_bf16(q), *args, dev(good[:, :7]), cu, dev(np.array([100, 10 ** 6], I32)), 0.125,
                                    True, torch.float32)
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_ERR_DEVICE
    w = paged.attention(paged.bf16_values(q), kc, ks, vc, vs, good, [0, 1, 2], [100, 112], 0.125, True)
    assert np.abs(L2[0].cpu().numpy() - w[1][0]).max() < 1e-3
    assert pkg.attn_last_device_status() == pkg.ATTN_OK


@gpu
def test_attention_repeats_bit_for_bit():
    rng = np.random.default_rng(24)
    kc, ks, vc, vs, table = _cache(rng, [5000, 100, 3000], 64, 2, 128)
    q = dev_bf16(_tokens(rng, 5, 8, 128, 0))
    g = [dev(a) for a in (kc, ks, vc, vs, table, np.array([0, 1, 4, 5], I32), np.array([5000, 100, 3000], I32))]
    first = pkg.attn_fwd_paged_fp8(q, *g, causal=True)
    for _ in range(5):
        again = pkg.attn_fwd_paged_fp8(q, *g, causal=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    ok()


# ------------------------------------------------------------------ together
@gpu
def test_a_servers_steps():
    """Prompts, then decoding steps, with requests that join late: tables, append and
    attention of every step against the plain forms of the three."""
    rng = np.random.default_rng(31)
    page, Hq, Hkv, d, R, width = 16, 4, 2, 64, 4, 12
    num_pages = 30
    kc, ks = np.zeros((num_pages, Hkv, page, d), np.uint8), np.ones((num_pages, Hkv), np.float32)
    vc, vs = kc.copy(), ks.copy()
    g = [dev(a) for a in (kc, ks, vc, vs)]
    table = np.zeros((R, width), I32)
    dtable = dev(table)
    free = rng.permutation(num_pages).astype(I32)
    lens = np.zeros(R, I32)
    for added in ([37, 0, 5, 16], [1, 0, 1, 1], [1, 50, 0, 1], [1, 1, 13, 1], [1, 1, 1, 1]):
        added = np.array(added, I32)
        T = int(added.sum()) + 2
        w = paged.tables(lens, added, free, table, page, T)
        kv, cu, slots, pos, taken = pkg.attn_kv_tables(dev(lens), dev(added), dev(free), dtable, page, T)
        kb, vb, qb = (_tokens(rng, T, H, d, 1) for H in (Hkv, Hkv, Hq))
        pkg.attn_kv_append_fp8(dev_bf16(kb), dev_bf16(vb), slots, *g)
        O, L = pkg.attn_fwd_paged_fp8(dev_bf16(qb), *g, dtable, cu, kv, causal=True, out_dtype=torch.float32)
        ok()
        table, lens = w[0].astype(I32), w[1].astype(I32)
        assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(slots.cpu().numpy(), w[3])
        kc, ks = paged.append(paged.bf16_values(kb), w[3], kc, ks)
        vc, vs = paged.append(paged.bf16_values(vb), w[3], vc, vs)
        Or, Lr, A, B = paged.attention(paged.bf16_values(qb), kc, ks, vc, vs, table, w[2], lens,
                                       float(np.float32(1 / np.sqrt(d))), True)
        n = int(w[2][-1])
        tol_o, tol_l = paged.bounds(Or, Lr, A, B, d, False)
        assert (np.abs(O.double().cpu().numpy() - Or)[:n] <= tol_o[:n]).all()
        assert (np.abs(L.double().cpu().numpy() - Lr)[:n] <= tol_l[:n]).all()
        free = free[int(w[5][0]):]


@gpu
def test_a_step_captured_and_replayed():
    """Tables, append and attention in one graph, replayed with other lengths."""
    rng = np.random.default_rng(32)
    page, Hq, Hkv, d, R, T = 32, 8, 2, 128, 3, 3
    lens = [np.array(x, I32) for x in ([100, 31, 64], [40, 200, 5])]
    kc, ks, vc, vs, table = _cache(rng, [210, 210, 210], page, Hkv, d)
    table = np.where(table < 0, 0, table)
    q, k, v = (dev_bf16(_tokens(rng, T, H, d, 0)) for H in (Hq, Hkv, Hkv))
    start = [dev(a) for a in (kc, ks, vc, vs)]
    g = [x.clone() for x in start]
    cached, added, free = dev(lens[0]), dev(np.ones(3, I32)), dev(np.arange(kc.shape[0] - 3, kc.shape[0], dtype=I32))
    tb = dev(table)
    ws = torch.empty(pkg.attn_fwd_paged_workspace_size(R, T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")

    def step():
        kv, cu, slots, _, _ = pkg.attn_kv_tables(cached, added, free, tb, page, T)
        pkg.attn_kv_append_fp8(k, v, slots, *g)
        return pkg.attn_fwd_paged_fp8(q, *g, tb, cu, kv, causal=True, workspace=ws)

    def reset(n):
        for x, y in zip(g, start):
            x.copy_(y)
        tb.copy_(dev(table))
        cached.copy_(dev(lens[n]))

    want = []
    for n in (0, 1):
        reset(n)
        want.append([x.clone() for x in (*step(), *g)])
    reset(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in (0, 1, 0):
        reset(n)
        graph.replay()
        ok()
        for a, b in zip((*out, *g), want[n]):
            assert torch.equal(a, b)


@gpu
def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(33)
    data = []
    for lens in ([3000, 50], [700, 900]):
        c = _cache(rng, lens, 64, 2, 64)
        q = dev_bf16(_tokens(rng, 2, 4, 64, 0))
        data.append((q, *[dev(a) for a in (*c, np.array([0, 1, 2], I32), np.asarray(lens, I32))]))
    want = [pkg.attn_fwd_paged_fp8(*x, causal=True) for x in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = []
    for _ in range(8):
        for x, s in zip(data, streams):
            with torch.cuda.stream(s):
                got.append(pkg.attn_fwd_paged_fp8(*x, causal=True))
    ok()
    for i, x in enumerate(got):
        assert torch.equal(x[0], want[i % 2][0]) and torch.equal(x[1], want[i % 2][1])


# ------------------------------------------------------------------ NaN where a row does not look
@gpu
@pytest.mark.parametrize("lens,news,Hq,Hkv,page", [([70, 33], [4, 3], 2, 1, 16), ([70, 300], [7, 9], 8, 2, 32),
                                                   ([700, 300], [40, 100], 4, 2, 64), ([500], [300], 1, 1, 128)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_attention_nan_values_reach_only_the_rows_that_see_them(lens, news, Hq, Hkv, page, d, out):
    """V holds NaN in some columns of the last tokens: a row before them must not
    meet it (0 * NaN), a row that sees them must."""
    rng = np.random.default_rng(sum(lens) + d)
    kc, ks, vc, vs, table = _cache(rng, lens, page, Hkv, d)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(I32)
    T = int(cu[-1])
    where = []
    for r, n in enumerate(lens):
        for back in (1, 2, min(news[r], 3)):
            key = n - back
            cols = rng.choice(d, 3, replace=False)
            vc[table[r, key // page], :, key % page, cols] = 0x7F if back % 2 else 0xFF
            where.append((r, key, cols))
    q = _tokens(rng, T, Hq, d, 0)
    g = [dev(a) for a in (kc, ks, vc, vs, table, cu, np.asarray(lens, I32))]
    O, L = pkg.attn_fwd_paged_fp8(dev_bf16(q), *g, None, True, out)
    ok()
    want = np.zeros((T, Hq, d), bool)
    for r, key, cols in where:
        for i in range(news[r]):
            if key <= lens[r] - news[r] + i:
                want[cu[r] + i][:, cols] = True
    assert np.array_equal(torch.isnan(O).cpu().numpy(), want)
    assert torch.isfinite(L).all()
    clean = vc.copy()
    clean[(clean & 0x7F) == 0x7F] = 0
    Or, _, A, B = paged.attention(paged.bf16_values(q), kc, ks, clean, vs, table, cu, lens,
                                  float(np.float32(1 / np.sqrt(d))), True)
    tol, _ = paged.bounds(Or, np.zeros(Or.shape[:2]), A, B, d, out == torch.bfloat16)
    err = np.abs(np.where(want, 0.0, O.double().cpu().numpy()) - np.where(want, 0.0, Or))
    assert (err <= tol).all()


@gpu
def test_attention_nan_in_keys_and_queries():
    rng = np.random.default_rng(41)
    for news in ([3], [40]):
        kc, ks, vc, vs, table = _cache(rng, [200], 32, 1, 64)
        kc[table[0, 199 // 32], 0, 199 % 32, 5] = 0x7F  # the last key: seen by the last query only
        T = news[0]
        q = _tokens(rng, T, 2, 64, 0)
        q[0, 1, 3] = 0x7FC0  # one query row is NaN
        q[1, 0, 3] = 0x7F80  # one has an infinity
        cu = np.array([0, T], I32)
        g = [dev(a) for a in (kc, ks, vc, vs, table, cu, np.array([200], I32))]
        O, L = pkg.attn_fwd_paged_fp8(dev_bf16(q), *g, None, True, torch.float32)
        ok()
        bad = np.zeros((T, 2), bool)
        bad[T - 1] = bad[0, 1] = bad[1, 0] = True
        assert np.array_equal(torch.isnan(L).cpu().numpy(), bad)
        assert np.array_equal(torch.isnan(O).all(-1).cpu().numpy(), bad)
        assert np.array_equal(torch.isnan(O).any(-1).cpu().numpy(), bad)
