"""The paged cache where its kernels could give each other different answers:
infinite queries, the smallest V scales, and ragged batches of more than 32
requests in every kernel, against the plain 64-bit implementation."""

import numpy as np
import pytest
import torch

import exact_attention_95_gb300 as pkg

import paged
from test_paged_cache import I32, _cache, _check_attention, dev, dev_bf16, ok

gpu = pytest.mark.gpu

# What a call runs: new tokens of two requests, heads of a kv head, columns of the table behind the last page.
KERNELS = {"8 rows, clusters": ([1, 1], 2, 0), "8 rows, ranges": ([1, 1], 2, 700), "16 rows": ([5, 4], 2, 0),
           "256 rows": ([40, 50], 1, 0), "both": ([5, 50], 2, 0)}


# ------------------------------------------------------------------ infinite queries
@gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("keys", [1, 3, 150])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("d", [64, 128])
def test_an_infinite_query_makes_its_row_nan_whatever_the_keys_signs(kernel, keys, sign, d):
    """Every key has a code of one sign in the infinite column, so that all logits are
    +inf or all -inf; a row that sees no key stays as such rows are."""
    news, G, extra = KERNELS[kernel]
    page, Hkv = 16, 2
    rng = np.random.default_rng(keys + d)
    kc, ks, vc, vs, table = _cache(rng, [keys, keys], page, Hkv, d, width_extra=1 + extra)
    kc[..., 3] = 0x38
    cu = np.concatenate([[0], np.cumsum(news)]).astype(I32)
    T, Hq = int(cu[-1]), G * Hkv
    q = paged.bf16_bits(rng.standard_normal((T, Hq, d)).astype(np.float32))
    bits = q.copy()
    inf = np.zeros((T, Hq), bool)
    for r in range(2):
        for t in (cu[r], cu[r + 1] - 1):  # (the first sees no key where there are more queries)
            inf[t, r] = inf[t, Hq - 1] = True
    bits[inf, 3] = 0x7F80 if sign > 0 else 0xFF80
    q[inf] = 0
    g = [dev(a) for a in (kc, ks, vc, vs, table, cu, np.array([keys, keys], I32))]
    for causal in (True, False):
        O, L = pkg.attn_fwd_paged_fp8(dev_bf16(bits), *g, None, causal, torch.float32)
        ok()
        Or, Lr, A, B = paged.attention(paged.bf16_values(q), kc, ks, vc, vs, table, cu, [keys, keys],
                                       float(np.float32(1 / np.sqrt(d))), causal)
        Og, Lg = O.double().cpu().numpy(), L.double().cpu().numpy()
        none = np.isneginf(Lr)
        assert np.array_equal(np.isnan(Lg), inf & ~none)
        assert np.isnan(Og[inf & ~none]).all()
        assert np.isneginf(Lg[none]).all() and (Og[none] == 0.0).all()
        rest = ~inf & ~none
        tol_o, tol_l = paged.bounds(Or, Lr, A, B, d, False)
        assert (np.abs(Og[rest] - Or[rest]) <= tol_o[rest]).all()
        assert (np.abs(Lg[rest] - Lr[rest]) <= tol_l[rest]).all()


# ------------------------------------------------------------------ the smallest V scales
@gpu
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
def test_values_at_the_smallest_scale_are_not_lost(kernel, d):
    """V = 448 * 2^-126 everywhere (the append's smallest scale): every row's O is V.

    A weight is off by 2^-11 at most.  Sums times the V scale and 1 / l are normal numbers
    or the result's own size."""
    news, G, extra = KERNELS[kernel]
    page, Hkv, lens = 32, 1, [50, 50]
    rng = np.random.default_rng(d)
    kc, ks, vc, vs, table = _cache(rng, lens, page, Hkv, d, width_extra=1 + extra)
    vc[:], vs[:] = 0x7E, 2.0 ** -126
    cu = np.concatenate([[0], np.cumsum(news)]).astype(I32)
    q = paged.bf16_bits(rng.standard_normal((int(cu[-1]), G * Hkv, d)).astype(np.float32))
    g = [dev(a) for a in (kc, ks, vc, vs, table, cu, np.array(lens, I32))]
    O, _ = pkg.attn_fwd_paged_fp8(dev_bf16(q), *g, None, True, torch.float32)
    ok()
    got = O.double().cpu().numpy() / (448.0 * 2.0 ** -126)
    assert np.abs(got - 1.0).max() <= 2.0 ** -11 + 2.0 ** -15


# ------------------------------------------------------------------ many requests
@gpu
@pytest.mark.parametrize("name,R,counts,Hq,Hkv,d,page", [
    # Few rows and many in one call, idle requests among them: both kernels' walks over groups of 32 requests.
    ("mixed", 70, (0, 1, 2, 9, 40, 150), 4, 2, 64, 16),
    ("mixed", 70, (0, 1, 2, 9, 40, 150), 2, 2, 128, 64),
    ("mixed, two of the tables' blocks", 1100, (0, 1, 2, 3, 33), 2, 1, 64, 32),
    # Up to 32 rows of a kv head only: the wide kernel finds nothing.
    ("16 rows", 100, (1, 2, 3, 6), 8, 2, 128, 32),
    # More than 32 in each: the 16-row kernel finds nothing.
    ("256 rows", 45, (40, 77, 130), 1, 1, 128, 16),
    # Groups above eight heads: a decoding step with 16, and with 40 (the wide kernel alone).
    ("16 heads", 70, (0, 1), 32, 2, 128, 16),
    ("40 heads", 70, (0, 1), 40, 1, 64, 16),
])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_attention_of_more_than_32_requests_in_every_kernel(name, R, counts, Hq, Hkv, d, page, out):
    rng = np.random.default_rng(R + d + Hq)
    news = rng.choice(counts, R)
    news[R // 2] = max(counts)
    lens = np.where(rng.random(R) < 0.1, 0, news + rng.integers(0, 300, R))
    _check_attention(rng, lens, news, Hq, Hkv, d, page, True, out, pad=3)


@gpu
@pytest.mark.parametrize("R,tall,Hq,Hkv,d", [(256, 128, 8, 2, 128), (256, 200, 4, 4, 64), (40, 40, 8, 1, 64)])
@pytest.mark.parametrize("ones", [False, True])
def test_a_tall_chunk_among_idle_requests(R, tall, Hq, Hkv, d, ones):
    """No more tokens than requests, most of them one request's: tiles of eight rows only."""
    rng = np.random.default_rng(R + tall + d)
    news = np.zeros(R, int)
    news[R // 3] = tall
    if ones:
        news[R // 2:R // 2 + R - tall] = 1
    assert news.sum() <= R
    lens = np.where(news > 0, news + rng.integers(0, 400, R), rng.integers(0, 50, R))
    _check_attention(rng, lens, news, Hq, Hkv, d, 16, True, torch.float32)


@gpu
@pytest.mark.parametrize("tall", [0, 50])
def test_the_largest_number_of_requests(tall):
    """16384 requests of up to 60 keys: a decoding step with some idle, and one with a tall chunk too."""
    R = 16384
    rng = np.random.default_rng(R + tall)
    news = (rng.random(R) < 0.9).astype(int)
    lens = rng.integers(0, 60, R)
    if tall:
        news[:] = 1
        news[R - 3], lens[R - 3] = tall, 300
    _check_attention(rng, lens, news, 2, 1, 64, 16, True, torch.float32)


@gpu
@pytest.mark.parametrize("R,pad,G,width", [(4, 2, 2, 0), (4, 2, 2, 700), (4, 9, 2, 0), (1, 90, 1, 0), (3, 2, 16, 0), (70, 70, 4, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_step_in_which_every_request_is_idle(R, pad, G, width, d):
    """Nothing is written, whichever kernels run."""
    rng = np.random.default_rng(R + pad)
    kc, ks, vc, vs, table = _cache(rng, [100] * R, 16, 2, d, width_extra=1 + width)
    g = [dev(a) for a in (kc, ks, vc, vs, table, np.zeros(R + 1, I32), np.full(R, 100, I32))]
    q = dev_bf16(paged.bf16_bits(rng.standard_normal((pad, 2 * G, d)).astype(np.float32)))
    O, L = torch.full_like(q, 7.0), torch.full((pad, 2 * G), 7.0, device="cuda")
    pkg.attn_fwd_paged_fp8(q, *g, None, True, O=O, LSE=L)
    ok()
    assert (O == 7).all() and (L == 7).all()


# ------------------------------------------------------------------ one workspace for several steps
def test_the_largest_of_the_steps_sizes_is_enough_for_each():
    """By the rule alone: sizes take two values for given heads and d, so that of one token
    more than requests is the largest for any R and T."""
    size = pkg.attn_fwd_paged_workspace_size
    for Hq, Hkv, d in ((8, 2, 128), (32, 2, 128), (4, 4, 64)):
        most = size(1, 2, Hq, Hkv, d)
        assert all(0 < size(R, T, Hq, Hkv, d) <= most for R in (1, 3, 256, 16384) for T in (1, 2, 4, 300, 20000))


@gpu
def test_one_workspace_through_steps_of_every_kind():
    """Many requests decode, then few take many tokens, then few decode: each in the same
    workspace, of the largest of the sizes, which holds what the step before left."""
    Hq, Hkv, d = 8, 2, 128
    steps = [([1] * 90, 90), ([5, 70], 2), ([1, 1], 2), ([4, 3, 2], 3), ([1] * 40, 40)]
    size = max(pkg.attn_fwd_paged_workspace_size(R, sum(n), Hq, Hkv, d) for n, R in steps)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(71)
    for news, R in steps:
        _check_attention(rng, [n + int(rng.integers(0, 900)) for n in news], news, Hq, Hkv, d, 32, True, workspace=ws)


# ------------------------------------------------------------------ waits
def test_the_waits_self_test_refuses_limits_out_of_range():
    for limit in (0, 10 ** 9 + 1, 2 ** 32):
        assert pkg.load_library().attn_selftest_paged_wait_timeout(limit, None) == pkg.ATTN_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("ms", [5, 50])
def test_a_wait_ends_at_its_limit_and_is_reported(ms):
    """The kernels' bounded wait on a barrier that nothing completes: a time, not a number of
    tries, so it is neither early nor late."""
    assert pkg.attn_selftest_paged_wait_timeout(10 ** 5) == pkg.ATTN_OK  # (the kernel's first launch loads it)
    assert pkg.attn_last_device_status() == pkg.ATTN_ERR_TIMEOUT
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    assert pkg.attn_selftest_paged_wait_timeout(ms * 10 ** 6) == pkg.ATTN_OK
    b.record()
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_ERR_TIMEOUT
    assert pkg.attn_last_device_status() == pkg.ATTN_OK
    assert 0.9 * ms <= a.elapsed_time(b) <= 2 * ms + 20  # (a try may take a while; launches beside it)
