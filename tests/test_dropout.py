"""Attention with dropout: the generator against published numbers, the masks bit for bit, and
forward and backward against the plain 64-bit implementation (tests/dropout.py) within
bounds derived there."""

import ctypes
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import exact_attention_95_gb300 as pkg
from exact_attention_95_gb300 import build as libbuild

import dropout as plain

gpu = pytest.mark.gpu
BAD, NO = pkg.ATTN_ERR_INVALID_ARG, pkg.ATTN_ERR_UNSUPPORTED
SEED = 0x1234567890ABCDEF


def _rng(seed=SEED, offset=3):
    seed = seed - 2 ** 64 if seed >= 2 ** 63 else seed
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def ok():
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK


def _make(seed, B, Hq, Hkv, N, d, q_mul=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(m * torch.randn(B, h, N, d, generator=g, device="cuda")).bfloat16()
            for h, m in ((Hq, q_mul), (Hkv, 1.0), (Hkv, 1.0), (Hq, 1.0))]


# ------------------------------------------------------------------ the generator (no GPU)
@pytest.mark.parametrize("rounds,c,k,want", [
    # Known answers published with the generator.
    (7, [0] * 4, [0] * 2, "5f6fb709 0d893f64 4f121f81 4f730a48"),
    (7, [plain.M32] * 4, [plain.M32] * 2, "5207ddc2 45165e59 4d8ee751 8c52f662"),
    (10, [0] * 4, [0] * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    (10, [plain.M32] * 4, [plain.M32] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    (10, [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0], "d16cfe09 94fdcceb 5001e420 24126ea1"),
])
def test_known_answers(rounds, c, k, want):
    got = plain.philox([torch.tensor(v) for v in c], [torch.tensor(v) for v in k], rounds)
    assert [int(x) for x in got] == [int(x, 16) for x in want.split()]


def test_the_numbers_are_uniform_and_independent():
    """Means of uniform numbers, of their products with shifted ones, and of single values: each
    within six standard deviations of what independent uniform numbers give."""
    u = plain.numbers(SEED, 0, 2, 3, 512).double()
    n = u.numel()
    x = (u - 127.5) / math.sqrt((256 ** 2 - 1) / 12)
    assert abs(x.mean()) < 6 / math.sqrt(n)
    for dims, shift in (((3,), (1,)), ((3,), (32,)), ((2,), (1,)), ((2, 3), (1, 1)), ((1,), (1,)), ((0,), (1,))):
        assert abs((x * x.roll(shift, dims)).mean()) < 6 / math.sqrt(n)
    for v in (0, 1, 127, 128, 255):
        assert abs((u == v).double().mean() * 256 - 1) < 6 * math.sqrt(256 / n)
    y = plain.numbers(SEED, 1, 2, 3, 512).double() - 127.5
    assert abs((x * y).mean()) / 74 < 6 / math.sqrt(n)


def test_plain_gradient_against_differences():
    torch.manual_seed(1)
    B, Hq, Hkv, N, d = 1, 4, 2, 9, 6
    Q, K, V, dO = (torch.randn(B, h, N, d).double() for h in (Hq, Hkv, Hkv, Hq))
    for causal in (False, True):
        r = plain.factors(SEED, 5, 0.3, B, Hq, N)
        args, scale = [Q, K, V], 0.4
        O = plain.forward(*args, r, scale, causal)[0]
        for i, (grad, _) in enumerate(plain.backward(*args, O, dO, r, scale, causal)):
            h, num = 1e-5, torch.zeros_like(grad)
            for e in range(grad.numel()):
                moved = []
                for sign in (1, -1):
                    a = [t.clone() for t in args]
                    a[i].view(-1)[e] += sign * h
                    moved.append((plain.forward(*a, r, scale, causal)[0] * dO).sum())
                num.view(-1)[e] = (moved[0] - moved[1]) / (2 * h)
            assert (grad - num).abs().max() < 1e-7


# ------------------------------------------------------------------ refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkg.load_library()


A = ctypes.c_void_p(0x10000)  # fake, aligned; never dereferenced on these paths
CASES = [
    (dict(Q=None), BAD), (dict(K=None), BAD), (dict(O=None), BAD), (dict(LSE=None), BAD), (dict(rng=None), BAD),
    (dict(V=ctypes.c_void_p(0x10008)), BAD), (dict(rng=ctypes.c_void_p(0x10004)), BAD), (dict(N=0), BAD),
    (dict(Hq=3, Hkv=2), BAD), (dict(scale=0.0), BAD), (dict(causal=2), BAD), (dict(d=96), NO), (dict(N=128 * 65536), NO),
    (dict(p=-0.1), BAD), (dict(p=1.0), BAD), (dict(p=float("nan")), BAD), (dict(p=0.9985), BAD), (dict(p=float("inf")), BAD),
]


@pytest.mark.parametrize("kw,want", CASES + [(dict(out=2), BAD)], ids=str)
def test_forward_refusals(lib, kw, want):
    a = dict(Q=A, K=A, V=A, O=A, LSE=A, rng=A, B=1, Hq=2, Hkv=1, N=128, d=64, scale=0.125, causal=0, p=0.1, out=0)
    a.update(kw)
    assert lib.attn_fwd_dropout(a["Q"], a["K"], a["V"], a["O"], a["LSE"], a["B"], a["Hq"], a["Hkv"], a["N"], a["d"],
                                a["scale"], a["causal"], a["p"], a["rng"], a["out"], None) == want


@pytest.mark.parametrize("kw,want", CASES + [(dict(ws=None), BAD), (dict(wsb=16), BAD), (dict(dQ=None), BAD),
                                             (dict(ws=ctypes.c_void_p(0x10080)), BAD)], ids=str)
def test_backward_refusals(lib, kw, want):
    a = dict(Q=A, K=A, V=A, O=A, dO=A, LSE=A, dQ=A, rng=A, B=1, Hq=2, Hkv=1, N=128, d=64, scale=0.125, causal=0, p=0.1,
             ws=A, wsb=1 << 40)
    a.update(kw)
    assert lib.attn_bwd_dropout(a["Q"], a["K"], a["V"], a["O"], a["dO"], a["LSE"], a["dQ"], A, A, a["B"], a["Hq"],
                                a["Hkv"], a["N"], a["d"], a["scale"], a["causal"], a["p"], a["rng"], a["ws"], a["wsb"],
                                None) == want


def test_binding_rejects_host_tensors(lib):
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        pkg.attn_fwd_dropout(x, x, x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        pkg.attn_bwd_dropout(x, x, x, x, x, torch.zeros(1, 2, 8), 0.1, torch.zeros(2, dtype=torch.int64))


# ------------------------------------------------------------------ masks, bit for bit
@gpu
@pytest.mark.parametrize("B,Hq,Hkv,N,d", [(1, 1, 1, 128, 128), (2, 3, 1, 33, 64), (1, 4, 2, 64, 128), (1, 2, 2, 1024, 128),
                                          (3, 2, 1, 500, 64), (1, 1, 1, 129, 64)])
@pytest.mark.parametrize("p,seed,offset", [(0.1, SEED, 3), (0.5, 0, 0), (0.99, 2 ** 64 - 1, 2 ** 32 - 1), (0.004, 5, 2 ** 40 + 9)])
def test_masks(B, Hq, Hkv, N, d, p, seed, offset):
    """Zero queries give every key the weight 1 / N, and V tells keys apart by column and power of two: an
    element of O is the sum of the kept keys' powers, whole in fp32, for both kernels of the forward.  The
    backward's mask: rows of dO with a column of their own, so that dV is zero where they drop a key."""
    r = plain.factors(seed, offset, p, B, Hq, N, "cuda")
    T = plain.threshold(p)
    kept = (r > 0).double()
    Q = torch.zeros(B, Hq, N, d, dtype=torch.bfloat16, device="cuda")
    K = torch.zeros(B, Hkv, N, d, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    j = torch.arange(N, device="cuda")
    per = min(16, -(-N // d))  # keys that share a column; 16 powers and a sum of them fit fp32
    V[:, :, j, j % d] = torch.exp2((j // d % 16).float()).bfloat16()
    assert per == -(-N // d)
    O, L = pkg.attn_fwd_dropout(Q, K, V, p, _rng(seed, offset), 1.0, False, torch.float32)
    ok()
    want = torch.zeros(B, Hq, N, d, dtype=torch.float64, device="cuda")
    want.index_add_(3, j % d, kept * torch.exp2((j // d).double()))
    got = O.double() * N * (1 - T / 256)
    assert torch.equal(torch.round(got), want) and (got - want).abs().max() < 0.1
    # dV_j = sum_i r_ij / N dO_i: with dO one column a row, of d rows and one head at a time (O = 0 keeps D out of it).
    for h in range(Hq):
        for i0 in range(0, N, d):
            dO = torch.zeros_like(Q)
            i = torch.arange(i0, min(i0 + d, N), device="cuda")
            dO[:, h, i, i - i0] = 1.0
            dV = pkg.attn_bwd_dropout(Q, K, V, torch.zeros_like(Q), dO, L, p, _rng(seed, offset), 1.0, False)[2]
            ok()
            want = torch.zeros(B, N, d, dtype=torch.bool, device="cuda")
            want[:, :, :len(i)] = kept[:, h, i].transpose(1, 2) > 0
            assert torch.equal(dV[:, h * Hkv // Hq] != 0, want)


# ------------------------------------------------------------------ forward and backward
SHAPES = [
    # B, Hq, Hkv, N, d
    (1, 1, 1, 1, 64), (2, 4, 2, 1, 128), (1, 8, 2, 31, 64), (1, 8, 2, 32, 128), (1, 8, 2, 33, 64),  # groups in one tile
    (2, 2, 2, 100, 128), (1, 4, 1, 100, 64), (1, 3, 3, 128, 64), (1, 2, 1, 129, 128), (1, 4, 2, 255, 64),
    (2, 4, 2, 257, 128), (1, 6, 2, 513, 128), (1, 16, 1, 650, 64), (1, 2, 2, 1000, 64), (2, 16, 4, 700, 128), (1, 2, 1, 2500, 128), (5, 40, 8, 520, 64),  # more key tiles than SMs
]


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("p", [0.1, 0.5, 0.97])
def test_forward_and_backward(shape, causal, p):
    B, Hq, Hkv, N, d = shape
    Q, K, V, dO = _make(N + d, *shape)
    scale, rng = 1 / math.sqrt(d), _rng(SEED + N, 7)
    r = plain.factors(SEED + N, 7, p, B, Hq, N, "cuda")
    Or, Lr, _, A, e = plain.forward(Q, K, V, r, scale, causal)
    for dtype in (torch.float32, torch.bfloat16):
        O, L = pkg.attn_fwd_dropout(Q, K, V, p, rng, scale, causal, dtype)
        ok()
        tol_o, tol_l = plain.forward_bounds(Or, Lr, A, e, dtype == torch.bfloat16)
        assert O.dtype == dtype and ((O.double() - Or).abs() <= tol_o).all(), (O.double() - Or).abs().max()
        assert ((L.double() - Lr).abs() <= tol_l).all()
        # A row all of whose kept keys are dropped is zero.
        empty = A.sum(-1) == 0
        assert (O[empty] == 0).all()
    grads = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, p, rng, scale, causal)
    ok()
    for name, got, (want, tol) in zip(("dQ", "dK", "dV"), grads, plain.backward(Q, K, V, O, dO, r, scale, causal)):
        assert ((got.double() - want).abs() <= tol).all(), (name, (got.double() - want).abs().max(), tol.max())


@gpu
def test_large_logits_and_rescaled_rows():
    """Logits of +-8 standard deviations, and keys that grow along the row so that its maximum keeps moving."""
    B, Hq, Hkv, N, d = 1, 4, 2, 900, 128
    Q, K, V, dO = _make(5, B, Hq, Hkv, N, d, q_mul=8.0)
    K = (K.float() * torch.linspace(0.2, 2.0, N, device="cuda")[:, None]).bfloat16()
    scale, rng, p = 1 / math.sqrt(d), _rng(11, 0), 0.2
    r = plain.factors(11, 0, p, B, Hq, N, "cuda")
    for causal in (False, True):
        Or, Lr, _, A, e = plain.forward(Q, K, V, r, scale, causal)
        O, L = pkg.attn_fwd_dropout(Q, K, V, p, rng, scale, causal)
        grads = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, p, rng, scale, causal)
        ok()
        tol_o, tol_l = plain.forward_bounds(Or, Lr, A, e, True)
        assert ((O.double() - Or).abs() <= tol_o).all() and ((L.double() - Lr).abs() <= tol_l).all()
        for got, (want, tol) in zip(grads, plain.backward(Q, K, V, O, dO, r, scale, causal)):
            assert ((got.double() - want).abs() <= tol).all()


@gpu
@pytest.mark.parametrize("N", [70, 600])
def test_probabilities_that_round_to_none_are_the_calls_without(N):
    Q, K, V, dO = _make(N, 1, 4, 2, N, 64)
    for p in (0.0, 0.0019):
        O, L = pkg.attn_fwd_dropout(Q, K, V, p, _rng(), None, True)
        O2, L2 = pkg.attn_fwd(Q, K, V, None, True)
        assert torch.equal(O, O2) and torch.equal(L, L2)
        a, b = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, p, _rng(), None, True), pkg.attn_bwd(Q, K, V, O, dO, L, None, True)
        ok()
        assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
        assert ((a[0] - b[0]).abs() <= 2 * plain.HALF * b[0].abs() + 1e-5).all()  # (dQ's sums have no fixed order)
    # The logsumexp is the one without dropout, bit for bit, whatever is dropped.
    assert torch.equal(pkg.attn_fwd_dropout(Q, K, V, 0.6, _rng(), None, True)[1], L2)
    ok()


@gpu
def test_calls_repeat_and_differ_by_seed_offset_and_head():
    Q, K, V, _ = _make(3, 1, 2, 2, 300, 64)
    Q[:, 1], K[:, 1], V[:, 1] = Q[:, 0], K[:, 0], V[:, 0]
    a = pkg.attn_fwd_dropout(Q, K, V, 0.3, _rng(1, 1))[0]
    assert torch.equal(a, pkg.attn_fwd_dropout(Q, K, V, 0.3, _rng(1, 1 + 2 ** 32))[0])
    assert not torch.equal(a[:, 0], a[:, 1])
    for other in (_rng(2, 1), _rng(1, 2), _rng(1 + 2 ** 32, 1), _rng(2 ** 63, 1)):
        assert not torch.equal(a, pkg.attn_fwd_dropout(Q, K, V, 0.3, other)[0])
    ok()


# ------------------------------------------------------------------ streams and graphs
@gpu
def test_streams_at_once():
    data = [(_make(i, 1, 4, 2, n, d), c) for i, (n, d, c) in enumerate([(1000, 128, True), (700, 64, False), (90, 128, True)])]
    want = []
    for (Q, K, V, dO), c in data:
        O, L = pkg.attn_fwd_dropout(Q, K, V, 0.2, _rng(), None, c)
        want.append((O, L, *pkg.attn_bwd_dropout(Q, K, V, O, dO, L, 0.2, _rng(), None, c)))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    rng = _rng()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for ((Q, K, V, dO), c), s in zip(data, streams):
            O, L = pkg.attn_fwd_dropout(Q, K, V, 0.2, rng, None, c, stream=s)
            got.append((O, L, *pkg.attn_bwd_dropout(Q, K, V, O, dO, L, 0.2, rng, None, c, stream=s)))
    ok()
    for k, g in enumerate(got):
        w = want[k % len(data)]
        for i in (0, 1, 3, 4):
            assert torch.equal(g[i], w[i])


@gpu
def test_graphs_replayed_side_by_side_follow_their_numbers():
    """Two steps captured from one stream, replayed on two at once, with new numbers each time."""
    B, Hq, Hkv, N, d = 1, 8, 4, 1500, 128
    sets = [_make(20 + i, B, Hq, Hkv, N, d) for i in range(2)]
    rngs = [_rng(100 + i, 0) for i in range(2)]
    graphs, outs = [], []
    for (Q, K, V, dO), rng in zip(sets, rngs):
        pkg.attn_fwd_dropout(Q, K, V, 0.1, rng, None, True)  # (attributes are set outside the capture)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            O, L = pkg.attn_fwd_dropout(Q, K, V, 0.1, rng, None, True)
            grads = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, 0.1, rng, None, True)
            rng[1] += 1  # the next step's
        graphs.append(g)
        outs.append((O, L, *grads))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for step in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        ok()
        for i, (Q, K, V, dO) in enumerate(sets):
            assert int(rngs[i][1]) == step + 1
            O, L = pkg.attn_fwd_dropout(Q, K, V, 0.1, _rng(100 + i, step), None, True)
            grads = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, 0.1, _rng(100 + i, step), None, True)
            ok()
            assert torch.equal(O, outs[i][0]) and torch.equal(L, outs[i][1])
            assert torch.equal(grads[1], outs[i][3]) and torch.equal(grads[2], outs[i][4])


@gpu
@pytest.mark.parametrize("B,Hq,Hkv,N,d", [(1, 4, 2, 500, 128), (2, 2, 2, 100, 64), (4, 40, 40, 140, 64)])
def test_steps_with_nothing_between_the_calls(B, Hq, Hkv, N, d):
    """Each call overwrites what the call before it reads or writes (keys and values become the last step's
    gradients, rotated; one workspace), and starts while that one ends: the bits are those of calls one at a time.
    (dQ, whose sums have no fixed order, goes nowhere.)"""
    Q, K0, V0, dO = _make(9, B, Hq, Hkv, N, d)
    freqs, _ = pkg.attn_rope_freqs(d)
    rng = _rng(4, 0)
    ws = torch.empty(pkg.attn_bwd_dropout_workspace_size(B, Hq, Hkv, N, d, True), dtype=torch.uint8, device="cuda")

    def run(wait):
        K, V, dQ = K0.clone(), V0.clone(), torch.empty_like(Q)
        dK, dV, O, L = torch.empty_like(K), torch.empty_like(K), torch.empty_like(Q), torch.empty(B, Hq, N, device="cuda")
        seen = []
        torch.cuda.synchronize()
        calls = [lambda: pkg.attn_fwd_dropout(Q, K, V, 0.2, rng, None, True, O=O, LSE=L),
                 lambda: pkg.attn_bwd_dropout(Q, K, V, O, dO, L, 0.2, rng, None, True, dQ, dK, dV, ws),
                 lambda: pkg.attn_rope_bwd(dK, dV, freqs, dQ_out=K, dK_out=V, amplitude=4.0),
                 lambda: pkg.attn_rope(K, None, freqs, Q_out=K)]
        for _ in range(12):
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()
            seen += [O.clone(), L.clone()]
        torch.cuda.synchronize()
        return seen + [K, V, dK, dV]

    want = run(True)
    assert all(torch.isfinite(t).all() for t in want)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
    ok()


@gpu
@pytest.mark.parametrize("module", [True, False])
def test_what_python_refuses(module, monkeypatch):
    if not module:
        monkeypatch.setattr(pkg, "_fast", False)
    Q, K, V, dO = _make(1, 1, 2, 2, 8, 64)
    L = torch.zeros(1, 2, 8, device="cuda")
    for exc, rng, p, kw in [
        (TypeError, None, 0.1, {}), (TypeError, torch.zeros(2, device="cuda"), 0.1, {}),
        (ValueError, torch.zeros(3, dtype=torch.int64, device="cuda"), 0.1, {}),
        (TypeError, torch.zeros(2, dtype=torch.int64), 0.1, {}), (pkg.AttnError, _rng(), 1.0, {}),
        (pkg.AttnError, _rng(), -0.5, {}),
    ]:
        with pytest.raises(exc):
            pkg.attn_fwd_dropout(Q, K, V, p, rng, **kw)
        with pytest.raises(exc):
            pkg.attn_bwd_dropout(Q, K, V, Q, dO, L, p, rng, **kw)
    with pytest.raises(TypeError):
        pkg.attn_fwd_dropout(Q.float(), K, V, 0.1, _rng())
    with pytest.raises(ValueError):
        pkg.attn_fwd_dropout(Q, K, V, 0.1, _rng(), O=torch.empty_like(Q[:, :1]))
    with pytest.raises(ValueError):
        pkg.attn_bwd_dropout(Q, K, V, Q, dO, L, 0.1, _rng(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    ok()


@gpu
@pytest.mark.parametrize("N", [40, 300])
def test_the_calls_give_the_same_without_the_module(N, monkeypatch):
    Q, K, V, dO = _make(N, 2, 6, 2, N, 64)
    ws = torch.empty(pkg.attn_bwd_dropout_workspace_size(2, 6, 2, N, 64, True), dtype=torch.uint8, device="cuda")
    got = []
    for module in (True, False):
        if not module:
            monkeypatch.setattr(pkg, "_fast", False)
        given = torch.empty_like(Q)
        O, L = pkg.attn_fwd_dropout(Q, K, V, 0.3, _rng(), 0.2, True, O=given)
        O32, _ = pkg.attn_fwd_dropout(Q, K, V, 0.3, _rng(), None, False, torch.float32)
        _, dK, dV = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, 0.3, _rng(), 0.2, True, workspace=ws)
        assert O is given
        got.append((O, L, O32, dK, dV))
    ok()
    assert all(torch.equal(a, b) for a, b in zip(*got))


FIRST = """
import torch
import exact_attention_95_gb300 as pkg
B, Hq, Hkv, N, d = 1, 4, 2, %d, %d
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g, device="cuda").bfloat16()
q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
v = x[:, :, Hq + Hkv:].transpose(1, 2).contiguous()
dO = torch.randn(B, Hq, N, d, generator=g, device="cuda").bfloat16()
freqs, _ = pkg.attn_rope_freqs(d)
rng = torch.tensor([3, 4], device="cuda")
def step():
    Q, K = pkg.attn_rope(q, k, freqs)
    O, L = pkg.attn_fwd_dropout(Q, K, v, 0.1, rng, None, True)
    dQ, dK, dV = pkg.attn_bwd_dropout(Q, K, v, O, dO, L, 0.1, rng, None, True)
    gq, gk = pkg.attn_rope_bwd(dQ, dK, freqs)
    return Q, K, O, L, dV, gk
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
want = step()
torch.cuda.synchronize()
assert pkg.attn_last_device_status() == pkg.ATTN_OK
assert all(torch.equal(a, b) for a, b in zip(got, want)) and float(got[2].float().abs().max()) > 0
print("captured first")
"""


@gpu
@pytest.mark.parametrize("N,d", [(90, 64), (600, 128)])
def test_the_first_calls_of_a_process_inside_a_capture(N, d):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % (N, d)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


@gpu
def test_threads_with_a_stream_each():
    data = [_make(30 + i, 1, 4, 2, 300 + 100 * i, 64) for i in range(4)]
    rng = _rng()

    def one(Q, K, V, dO):
        O, L = pkg.attn_fwd_dropout(Q, K, V, 0.4, rng, None, True)
        _, dK, dV = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, 0.4, rng, None, True)
        return O, L, dK, dV

    want = [one(*d) for d in data]
    torch.cuda.synchronize()
    got = [None] * len(data)

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got[i] = one(*data[i])
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


# ------------------------------------------------------------------ a layer's step
@gpu
@pytest.mark.parametrize("B,Hq,Hkv,N,d,rot,interleaved", [(2, 6, 2, 333, 128, 64, False), (1, 4, 4, 90, 64, 64, True)])
def test_a_training_step(B, Hq, Hkv, N, d, rot, interleaved):
    """Positions, attention with dropout, its backward and the positions' gradient into the projection's:
    each call on what the one before gave, checked against 64 bits."""
    import positions as pos64
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g, device="cuda").bfloat16()
    dx = torch.full_like(x, float("nan"))

    def part(t, a, b):
        return t[:, :, a:b].transpose(1, 2)

    freqs, amplitude = pkg.attn_rope_freqs(rot, scaling="linear", factor=2.0)
    p, rng = 0.15, _rng(77, 2)
    Q, K = pkg.attn_rope(part(x, 0, Hq), part(x, Hq, Hq + Hkv), freqs, None, interleaved, amplitude)
    V = part(x, Hq + Hkv, Hq + 2 * Hkv).contiguous()
    O, L = pkg.attn_fwd_dropout(Q, K, V, p, rng, None, True)
    dO = torch.randn(B, Hq, N, d, generator=g, device="cuda").bfloat16()
    dQ, dK, dV = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, p, rng, None, True)
    pkg.attn_rope_bwd(dQ, dK, freqs, None, interleaved, amplitude, part(dx, 0, Hq), part(dx, Hq, Hq + Hkv))
    part(dx, Hq + Hkv, Hq + 2 * Hkv).copy_(dV)
    ok()

    def rows(t):
        return t.transpose(1, 2).reshape(B * N, t.shape[1], d).double().cpu().numpy()

    def turned(got, src, sign):
        y, size = pos64.rotate(rows(src), list(range(N)) * B, freqs.tolist(), interleaved, amplitude, sign)
        assert (abs(rows(got) - y) <= pos64.tolerance(y, size, True)).all()

    scale = 1 / math.sqrt(d)
    r = plain.factors(77, 2, p, B, Hq, N, "cuda")
    turned(Q, part(x, 0, Hq), 1.0)
    turned(K, part(x, Hq, Hq + Hkv), 1.0)
    Or, Lr, _, A, e = plain.forward(Q, K, V, r, scale, True)
    tol_o, tol_l = plain.forward_bounds(Or, Lr, A, e, True)
    assert ((O.double() - Or).abs() <= tol_o).all() and ((L.double() - Lr).abs() <= tol_l).all()
    for got, (want, tol) in zip((dQ, dK, dV), plain.backward(Q, K, V, O, dO, r, scale, True)):
        assert ((got.double() - want).abs() <= tol).all()
    turned(part(dx, 0, Hq), dQ, -1.0)
    turned(part(dx, Hq, Hq + Hkv), dK, -1.0)
    assert torch.isfinite(dx).all()
