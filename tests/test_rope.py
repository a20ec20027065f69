"""Rotary positions on the GPU against the plain 64-bit implementation
(tests/positions.py), within bounds derived there: layouts, types, strides and
positions; their gradient; the paged append that applies them; and the calls as a
layer strings them together."""

import math

import numpy as np
import pytest
import torch

import exact_attention_95_gb300 as pkg

import paged
import positions as pos64
from test_paged_cache import I32, dev, ok

gpu = pytest.mark.gpu
pytestmark = gpu
FAR = 2 ** 31 - 1


def _f64(t):
    return t.double().cpu().numpy()


def _rand(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _rows(t):
    """[rows, H, d] float64 of a [T, H, d] or [B, H, N, d] tensor, by batch and token."""
    x = _f64(t)
    return x if x.ndim == 3 else x.transpose(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])


def _check(got, X, positions, freqs, interleaved, amplitude, sign=1.0):
    y, size = pos64.rotate(_rows(X), positions, freqs.tolist(), interleaved, amplitude, sign)
    tol = pos64.tolerance(y, size, X.dtype == torch.bfloat16)
    g = _rows(got)
    assert got.dtype == X.dtype and got.shape == X.shape
    assert (np.abs(g - y) <= tol).all(), np.abs(g - y).max()
    assert np.array_equal(g[size == 0.0], y[size == 0.0])  # what does not turn stays


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 80)])
def test_angles_at_every_distance(d, rot, dtype, interleaved):
    """Unit vectors show cos and sin themselves, at positions up to the last."""
    freqs, amplitude = pkg.attn_rope_freqs(rot)
    positions = np.array([0, 1, 2, 7, 1000, 4095, 131071, 2 ** 24 + 1, FAR - 1, FAR, -1, -FAR], I32)
    X = torch.zeros(len(positions), 2, d, dtype=dtype, device="cuda")
    X[:, 0, 0:rot:2] = 1.0
    X[:, 1, 1:rot:2] = -1.0
    X[:, :, rot:] = 3.0
    Y, none = pkg.attn_rope(X, None, freqs, dev(positions), interleaved)
    Z, _ = pkg.attn_rope_bwd(X, None, freqs, dev(positions), interleaved)
    ok()
    assert none is None
    _check(Y, X, positions, freqs, interleaved, 1.0)
    _check(Z, X, positions, freqs, interleaved, 1.0, -1.0)


@pytest.mark.parametrize("interleaved,dtype", [(False, torch.bfloat16), (True, torch.bfloat16), (False, torch.float32),
                                               (True, torch.float32)])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", [(1, 1, 1, 1, 64, 64), (2, 33, 3, 1, 128, 128), (3, 257, 6, 2, 64, 32),
                                              (1, 1000, 32, 8, 128, 128), (5, 17, 40, 5, 128, 96)])
@pytest.mark.parametrize("where", ["start", "shared", "own"])
def test_heads_by_tokens(B, N, Hq, Hkv, d, rot, interleaved, dtype, where):
    """[B, H, N, d], contiguous and out of a packed projection, at positions 0.., shared or each batch's own."""
    freqs, amplitude = pkg.attn_rope_freqs(rot, scaling="parts", factor=4.0, original_len=1024)
    rng = np.random.default_rng(N)
    positions = {"start": None, "shared": rng.integers(-1, 200000, N).astype(I32),
                 "own": rng.integers(-1, 200000, (B, N)).astype(I32)}[where]
    flat = np.broadcast_to(np.arange(N) if positions is None else positions, (B, N)).reshape(-1)
    given = None if positions is None else dev(positions)
    packed = _rand(N + d, B, N, Hq + 2 * Hkv, d, dtype=dtype)
    Q, K = packed[:, :, :Hq].transpose(1, 2), packed[:, :, Hq:Hq + Hkv].transpose(1, 2)
    for q, k in ((Q, K), (Q.contiguous(), K.contiguous()), (Q, K.contiguous())):
        Qo, Ko = pkg.attn_rope(q, k, freqs, given, interleaved, amplitude)
        assert Qo.is_contiguous() and Ko.is_contiguous()
        dQ, dK = pkg.attn_rope_bwd(q, k, freqs, given, interleaved, amplitude)
        ok()
        _check(Qo, Q, flat, freqs, interleaved, amplitude)
        _check(Ko, K, flat, freqs, interleaved, amplitude)
        _check(dQ, Q, flat, freqs, interleaved, amplitude, -1.0)
        _check(dK, K, flat, freqs, interleaved, amplitude, -1.0)


@pytest.mark.parametrize("T,Hq,Hkv,d,rot", [(1, 1, 1, 128, 128), (64, 32, 8, 128, 128), (777, 16, 16, 64, 64), (3000, 6, 2, 64, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_tokens(T, Hq, Hkv, d, rot, interleaved):
    freqs, amplitude = pkg.attn_rope_freqs(rot, scaling="linear", factor=3.0)
    positions = np.random.default_rng(T).integers(-2, 10 ** 6, T).astype(I32)
    x = _rand(T, T, Hq + 2 * Hkv, d)
    Q, K = x[:, :Hq], x[:, Hq:Hq + Hkv]
    Qo, Ko = pkg.attn_rope(Q, K, freqs, dev(positions), interleaved, amplitude)
    ok()
    _check(Qo, Q, positions, freqs, interleaved, amplitude)
    _check(Ko, K, positions, freqs, interleaved, amplitude)
    Qo, _ = pkg.attn_rope(Q, K, freqs, None, interleaved, amplitude)
    ok()
    _check(Qo, Q, np.arange(T), freqs, interleaved, amplitude)


@pytest.mark.parametrize("rot", [128, 48])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_between_other_rows(rot, interleaved):
    """In a packed projection, in place and into another; V's rows and the array's ends stay as they were."""
    B, N, Hq, Hkv, d = 2, 65, 6, 2, 128
    freqs, _ = pkg.attn_rope_freqs(rot)
    positions = torch.arange(5, 5 + N, dtype=torch.int32, device="cuda")
    positions[3] = -1
    for bwd, f in ((False, pkg.attn_rope), (True, pkg.attn_rope_bwd)):
        x = _rand(7, B, N, Hq + 2 * Hkv, d)
        want = f(x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2), freqs, positions, interleaved)
        y = x.clone()
        q, k = y[:, :, :Hq].transpose(1, 2), y[:, :, Hq:Hq + Hkv].transpose(1, 2)
        got = f(q, k, freqs, positions, interleaved, Q_out=q, K_out=k) if not bwd else f(
            q, k, freqs, positions, interleaved, dQ_out=q, dK_out=k)
        ok()
        assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert torch.equal(y[:, :, Hq + Hkv:], x[:, :, Hq + Hkv:])
        # Contiguous heads back into slices of a packed array.
        z = torch.full_like(x, 9.0)
        f(*(t.contiguous() for t in (x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2))), freqs, positions,
          interleaved, 1.0, z[:, :, :Hq].transpose(1, 2), z[:, :, Hq:Hq + Hkv].transpose(1, 2))
        ok()
        assert torch.equal(z[:, :, :Hq + Hkv], y[:, :, :Hq + Hkv]) and (z[:, :, Hq + Hkv:] == 9.0).all()


def test_strides_of_single_rows_and_repeated_inputs():
    freqs, _ = pkg.attn_rope_freqs(64)
    x = _rand(3, 1, 64)
    Y, _ = pkg.attn_rope(x.expand(1, 5, 7, 64), None, freqs)  # one row for all heads and tokens
    ok()
    _check(Y, x.expand(1, 5, 7, 64), np.arange(7), freqs, False, 1.0)
    one = x.as_strided((1, 1, 1, 64), (3, 5, 7, 1))  # strides of nothing
    Y, _ = pkg.attn_rope(one, one, freqs, torch.tensor([9], dtype=torch.int32, device="cuda"))
    ok()
    _check(Y, one, [9], freqs, False, 1.0)
    assert pkg.attn_rope(x.new_empty(0, 4, 64), x.new_empty(0, 2, 64), freqs)[1].shape == (0, 2, 64)
    assert pkg.attn_rope(x.new_empty(2, 4, 0, 64), None, freqs)[0].shape == (2, 4, 0, 64)


def test_offsets_past_32_bits():
    """Batches of a few tokens 2^32 elements and more apart (8 GB), in place."""
    freqs, _ = pkg.attn_rope_freqs(128)
    far = 2 ** 32 + 256
    big = torch.empty(far + 8192, dtype=torch.bfloat16, device="cuda")
    X = big.as_strided((2, 3, 5, 128), (far, 128, 768, 1))
    X.copy_(_rand(8, 2, 3, 5, 128))
    was = X.clone()
    positions = torch.tensor([[1, 2, 3, 4, 5], [9, 8, 7, -1, 6]], dtype=torch.int32, device="cuda")
    Y, _ = pkg.attn_rope(X, None, freqs, positions, Q_out=X)
    ok()
    assert Y is X
    _check(X.contiguous(), was, positions.cpu().numpy().reshape(-1), freqs, False, 1.0)


def test_gradient_against_differences():
    """The rotation is linear: differences of any size have no error of their own.  Per element in
    fp32, off by twice what each of the two rotations may be."""
    B, H, N, d, rot = 1, 2, 9, 64, 32
    freqs, amplitude = pkg.attn_rope_freqs(rot, scaling="parts", factor=8.0, original_len=64)
    X, G = _rand(1, B, H, N, d, dtype=torch.float32), _rand(2, B, H, N, d, dtype=torch.float32)
    for interleaved in (False, True):
        grad = _f64(pkg.attn_rope_bwd(G, None, freqs, None, interleaved, amplitude)[0])
        base = _f64(pkg.attn_rope(X, None, freqs, None, interleaved, amplitude)[0])
        size = pos64.rotate(_rows(X), np.arange(N), freqs.tolist(), interleaved, amplitude)[1]
        for e in range(d):
            step = X.clone()
            step[..., e] += 1.0
            diff = _f64(pkg.attn_rope(step, None, freqs, None, interleaved, amplitude)[0]) - base
            want = (diff * _f64(G)).sum(-1)  # of sum(rope(x) * G) by x's element e, every row its own
            tol = 8 * pos64.TURN * (np.abs(size).max() + 2) * np.abs(_f64(G)).sum(-1)
            assert (np.abs(grad[..., e] - want) <= tol).all()
    ok()


def test_nan_and_infinity_stay_in_their_pairs():
    freqs, _ = pkg.attn_rope_freqs(128)
    for interleaved in (False, True):
        X = _rand(4, 3, 2, 128)
        X[1, 0, 10], X[2, 1, 67] = float("nan"), float("inf")
        Y, _ = pkg.attn_rope(X, None, freqs, torch.tensor([4, 5, 6], dtype=torch.int32, device="cuda"), interleaved)
        ok()
        pairs = {10: (10, 11), 67: (66, 67)} if interleaved else {10: (10, 74), 67: (3, 67)}
        bad = torch.zeros(3, 2, 128, dtype=torch.bool)
        bad[1, 0, list(pairs[10])] = True
        bad[2, 1, list(pairs[67])] = True
        assert torch.equal(~torch.isfinite(Y.cpu()), bad)


@pytest.mark.parametrize("module", [True, False])
def test_streams_graphs_and_the_module(module, monkeypatch):
    """On a stream of its own, captured and replayed on new numbers, with and without the extension module."""
    if not module:
        monkeypatch.setattr(pkg, "_fast", False)
    freqs, _ = pkg.attn_rope_freqs(64)
    Q, K = _rand(5, 2, 4, 100, 64), _rand(6, 2, 2, 100, 64)
    positions = torch.arange(100, dtype=torch.int32, device="cuda")
    want = pkg.attn_rope(Q, K, freqs, positions)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pkg.attn_rope(Q, K, freqs, positions, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.attn_rope(Q, K, freqs, positions, Q_out=outs[0], K_out=outs[1])
        pkg.attn_rope_bwd(outs[0], outs[1], freqs, positions, dQ_out=outs[0], dK_out=outs[1])
    positions += 1000
    Q.mul_(2)
    graph.replay()
    ok()
    there, back = pkg.attn_rope(Q, K, freqs, positions), None
    back = pkg.attn_rope_bwd(*there, freqs, positions)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(outs, back))


@pytest.mark.parametrize("module", [True, False])
def test_what_python_refuses(module, monkeypatch):
    if not module:
        monkeypatch.setattr(pkg, "_fast", False)
    freqs, _ = pkg.attn_rope_freqs(64)
    x, p = _rand(1, 5, 4, 64), torch.arange(5, dtype=torch.int32, device="cuda")
    for exc, args, kw in [
        (TypeError, (x.half(), None, freqs), {}), (ValueError, (x[0], None, freqs), {}),
        (TypeError, (x, x.float(), freqs), {}), (ValueError, (x, x[:4], freqs), {}),
        (TypeError, (x, x[None], freqs), {}), (ValueError, (x.transpose(1, 2), None, freqs), {}),
        (ValueError, (x[..., ::2], None, freqs[:16]), {}), (TypeError, (x, None, freqs.int()), {}),
        (ValueError, (x, None, torch.cat([freqs, freqs])), {}), (ValueError, (x, None, freqs[:0]), {}),
        (TypeError, (x, None, freqs.cpu()), {}), (TypeError, (x, None, freqs, p.long()), {}),
        (ValueError, (x, None, freqs, p[:4]), {}), (ValueError, (x, None, freqs, p[None]), {}),
        (TypeError, (x, None, freqs, p.cpu()), {}), (ValueError, (x, None, freqs, p), dict(K_out=x)),
        (TypeError, (x, None, freqs, p), dict(Q_out=x.float())), (ValueError, (x, None, freqs, p), dict(Q_out=x[:4])),
        (pkg.AttnError, (x, x, freqs, p), dict(Q_out=x)), (pkg.AttnError, (x, None, freqs, p, False, -1.0), {}),
        (pkg.AttnError, (x, None, freqs[:4], p), {}), (pkg.AttnError, (x, None, freqs, p), dict(Q_out=x[:1].expand(5, 4, 64))),
        (pkg.AttnError, (x.flatten()[1:257].view(1, 4, 64), None, freqs), {}),
    ]:
        with pytest.raises(exc):
            pkg.attn_rope(*args, **kw)
    ok()


# ------------------------------------------------------------------ the append
def _cache_for(rng, num_pages, Hkv, page, d):
    codes = [rng.integers(0, 255, (num_pages, Hkv, page, d)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 0x7F) == 0x7F] = 0x3A  # no NaN codes
    return codes, [2.0 ** rng.integers(-12, -4, (num_pages, Hkv)).astype(np.float32) for _ in range(2)]


def _append_case(rng, lens, page, extra):
    """Slots and positions of new tokens [cached, new] a request, with `extra` places behind them."""
    need = [-(-(c + n) // page) for c, n in lens]
    ids = rng.permutation(sum(need) + 2)
    slots, pos, at = [], [], 0
    for (c, n), k in zip(lens, need):
        row, at = ids[at:at + k], at + k
        for i in range(c, c + n):
            slots.append(int(row[i // page]) * page + i % page)
            pos.append(i)
    return np.array(slots + [-1] * extra, np.int64), np.array(pos + [-1] * extra, I32), sum(need) + 2


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 32), (128, 128), (128, 16), (128, 112)])
@pytest.mark.parametrize("lens,page,extra,Hq,Hkv", [
    ([(0, 1)], 16, 0, 1, 1), ([(5, 1), (16, 1), (31, 1)] * 5, 16, 3, 8, 2), ([(7, 3), (0, 4), (60, 8)], 64, 1, 6, 3),
    ([(10, 13), (3, 16), (100, 40)], 32, 0, 4, 4), ([(50, 300), (0, 1), (127, 2)], 128, 5, 4, 2),
    ([(30, 1500), (0, 70)], 64, 2, 2, 1),
])
def test_append_matches_the_plain_form(lens, page, extra, Hq, Hkv, d, rot, interleaved):
    rng = np.random.default_rng(len(lens) + page + d + rot)
    slots, positions, num_pages = _append_case(rng, lens, page, extra)
    T = len(slots)
    freqs, amplitude = pkg.attn_rope_freqs(rot, scaling="parts", factor=8.0, original_len=512)
    codes, scales = _cache_for(rng, num_pages, Hkv, page, d)
    x = _rand(T, T, Hq + 2 * Hkv, d) * torch.exp2(_rand(T + 1, T, 1, 1).float() * 2).bfloat16()
    Q, K, V = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cache = [dev(codes[0]), dev(scales[0]), dev(codes[1]), dev(scales[1])]
    Qo = pkg.attn_kv_append_rope_fp8(Q, K, V, dev(positions), dev(slots), freqs, *cache, interleaved, amplitude)
    ok()
    _check(Qo, Q, positions, freqs, interleaved, amplitude)
    assert Qo.is_contiguous()
    y, size = pos64.rotate(_f64(K), positions, freqs.tolist(), interleaved, amplitude)
    got = [c.cpu().numpy() for c in cache]
    pos64.check_append(y, size, slots, codes[0], scales[0], got[0], got[1])
    want = paged.append(_f64(V), slots, codes[1], scales[1])
    assert np.array_equal(got[2], want[0]) and np.array_equal(got[3].astype(np.float64), want[1])


def test_append_at_scales_that_are_no_power_of_two_and_of_tokens_without_positions():
    """Any scale above zero is a cache's; a token with a slot and no position is appended as it is."""
    rng = np.random.default_rng(5)
    page, d, H = 16, 64, 2
    lens = [(9, 1), (4, 9), (1, 15)]
    slots, positions, num_pages = _append_case(rng, lens, page, 0)
    positions[3::4] = -1
    codes, scales = _cache_for(rng, num_pages, H, page, d)
    scales = [np.where(np.arange(H) == 0, s * np.float32(1.37 * 64), s).astype(np.float32) for s in scales]
    freqs, _ = pkg.attn_rope_freqs(64)
    Q, K, V = (_rand(i, len(slots), H, d) for i in range(3))
    cache = [dev(codes[0]), dev(scales[0]), dev(codes[1]), dev(scales[1])]
    Qo = pkg.attn_kv_append_rope_fp8(Q, K, V, dev(positions), dev(slots), freqs, *cache, Q_out=Q)
    ok()
    assert Qo is Q
    y, size = pos64.rotate(_f64(K), positions, freqs.tolist(), False, 1.0)
    # (x / scale is rounded once more to fp32 here)
    pos64.check_append(y, size + 2.0 ** -2 * np.abs(y), slots, codes[0], scales[0], cache[0].cpu().numpy(), cache[1].cpu().numpy())


@pytest.mark.parametrize("new", [1, 9, 50])
def test_tokens_without_positions_keep_infinities_apart(new):
    """A key that is not rotated is appended as attn_kv_append_fp8 appends it, infinities and NaNs among its numbers."""
    page, d, H = 64, 64, 2
    freqs, _ = pkg.attn_rope_freqs(d)
    rng = np.random.default_rng(new)
    slots, positions, num_pages = _append_case(rng, [(2, new)], page, 0)
    codes, scales = _cache_for(rng, num_pages, H, page, d)
    K, V = _rand(1, new, H, d), _rand(2, new, H, d)
    K[0, 1, 3], K[new - 1, 0, 40] = float("inf"), float("nan")
    one, two = ([dev(codes[0]), dev(scales[0]), dev(codes[1]), dev(scales[1])] for _ in range(2))
    Qo = pkg.attn_kv_append_rope_fp8(K, K, V, dev(np.full(new, -1, I32)), dev(slots), freqs, *one)
    pkg.attn_kv_append_fp8(K, V, dev(slots), *two)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    assert torch.equal(Qo.view(torch.int16), K.view(torch.int16))


@pytest.mark.parametrize("new", [1, 6, 40])
def test_append_of_infinities_and_nans(new):
    """They reach no other pair's codes, and no scale."""
    page, d, H = 64, 128, 2
    freqs, _ = pkg.attn_rope_freqs(d)
    rng = np.random.default_rng(new)
    slots, positions, num_pages = _append_case(rng, [(3, new)], page, 0)
    codes, scales = _cache_for(rng, num_pages, H, page, d)
    K, V = _rand(1, new, H, d), _rand(2, new, H, d)
    clean = [dev(codes[0]), dev(scales[0]), dev(codes[1]), dev(scales[1])]
    dirty = [c.clone() for c in clean]
    K[0, 0, 5] = K[0, 0, 69] = 0.0
    V[new - 1, 1, 7] = 0.0
    pkg.attn_kv_append_rope_fp8(K, K, V, dev(positions), dev(slots), freqs, *clean)
    K[0, 0, 5], V[new - 1, 1, 7] = float("inf"), float("nan")
    pkg.attn_kv_append_rope_fp8(K, K, V, dev(positions), dev(slots), freqs, *dirty)
    ok()
    p, off = int(slots[0]) // page, int(slots[0]) % page
    q, last = int(slots[-1]) // page, int(slots[-1]) % page
    for a, b in zip(clean, dirty):
        if a.dtype == torch.float32:
            assert torch.equal(a, b)
    for i, at in ((0, [(p, 0, off, 5), (p, 0, off, 69)]), (2, [(q, 1, last, 7)])):
        diff = (clean[i] != dirty[i]).nonzero().tolist()
        assert sorted(map(tuple, diff)) == sorted(at)
        assert all(int(dirty[i][k]) & 0x7F in (0x7E, 0x7F) for k in at)


def test_append_on_a_border_of_the_scales():
    """448 * 2^k fits a scale of 2^k, the next larger fp32 number does not: with rotations by whole quarter turns
    the numbers are exact but for the rounding of a zero."""
    freqs = torch.zeros(32, dtype=torch.int64, device="cuda")
    for k, v, want in ((0, 448.0, 1.0), (0, 450.0, 2.0), (0, 446.0, 1.0), (0, 2.0 ** -140, 2.0 ** -126), (0, 0.0, 2.0 ** -126)):
        K = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
        K[0, 0, 3] = v
        cache = [c for _ in range(2) for c in (torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device="cuda"),
                                               torch.ones(1, 1, device="cuda"))]
        pkg.attn_kv_append_rope_fp8(K, K, K, torch.tensor([5], dtype=torch.int32, device="cuda"),
                                    torch.zeros(1, dtype=torch.int64, device="cuda"), freqs, *cache)
        ok()
        assert float(cache[1]) == want and float(cache[3]) == want, v


@pytest.mark.parametrize("module", [True, False])
def test_a_servers_steps_with_rotated_keys(module, monkeypatch):
    """Tables, append and attention, step after step: against attention in 64 bits over what the pages hold, the
    queries being those that the append returned; and the same bits with the calls strung together in a graph."""
    if not module:
        monkeypatch.setattr(pkg, "_fast", False)
    page, Hq, Hkv, d, rot, R = 32, 8, 2, 128, 64, 3
    freqs, amplitude = pkg.attn_rope_freqs(rot, scaling="linear", factor=2.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    free = torch.randperm(40, generator=g, device="cuda").int()
    table = torch.zeros(R, 12, dtype=torch.int32, device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    cache = [x for _ in range(2) for x in (torch.zeros(40, Hkv, page, d, dtype=torch.uint8, device="cuda"),
                                           torch.ones(40, Hkv, device="cuda"))]
    for news in ([70, 1, 130], [1, 1, 1], [1, 0, 5]):
        T = sum(news) + 2
        x = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device="cuda").bfloat16()
        Q, K, V = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        before = [c.clone() for c in (table, *cache)]
        added = torch.tensor(news, dtype=torch.int32, device="cuda")

        def step(lens_in, table, cache, O, L):
            lens, cu, slots, pos, taken = pkg.attn_kv_tables(lens_in, added, free, table, page, T)
            Qr = pkg.attn_kv_append_rope_fp8(Q, K, V, pos, slots, freqs, *cache, True, amplitude)
            pkg.attn_fwd_paged_fp8(Qr, *cache, table, cu, lens, causal=True, out_dtype=torch.float32, O=O, LSE=L)
            return lens, cu, taken, Qr

        O, L = torch.zeros(T, Hq, d, device="cuda"), torch.zeros(T, Hq, device="cuda")
        old = lens
        lens, cu, taken, Qr = step(lens, table, cache, O, L)
        ok()
        used = sum(news)
        Or, Lr, A, B = paged.attention(_f64(Qr), *(c.cpu().numpy() for c in cache), table.cpu().numpy(), cu.tolist(),
                                       lens.tolist(), 1 / math.sqrt(d), True)
        tol_o, tol_l = paged.bounds(Or, Lr, A, B, d, False)
        assert (np.abs(_f64(O) - Or)[:used] <= tol_o[:used]).all() and (np.abs(_f64(L) - Lr)[:used] <= tol_l[:used]).all()
        assert torch.equal(Qr[used:], Q[used:]) and (O[used:] == 0).all()
        # The same in a graph, from the same start.
        again, O2, L2 = [c.clone() for c in before], torch.zeros_like(O), torch.zeros_like(L)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            kept = step(old, again[0], again[1:], O2, L2)
        graph.replay()
        ok()
        assert torch.equal(O, O2) and torch.equal(L, L2) and torch.equal(kept[3], Qr)
        assert all(torch.equal(a, b) for a, b in zip(again, (table, *cache)))
        free = free[int(taken[0]):].contiguous()
