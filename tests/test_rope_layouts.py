"""Rotary positions in place and between other rows of packed arrays of any order: whether two sets of rows share an
element (csrc/checks.h, compiled for the host) against their elements one by one, refusals, and
the rotation itself."""

import os
import random
import subprocess

import numpy as np
import pytest
import torch

import exact_attention_95_gb300 as pkg
from exact_attention_95_gb300 import build as libbuild

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_95_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "checks.h"
int main() {
  long long p[2], n[2][3], s[2][3], d;
  while (std::scanf("%lld", &d) == 1) {
    for (int i = 0; i < 2; ++i)
      if (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &p[i], &n[i][0], &n[i][1], &n[i][2], &s[i][0], &s[i][1], &s[i][2]) != 7)
        return 1;
    attn::Rows r[2] = {{(void*)p[0], n[0][0], n[0][1], n[0][2], s[0][0], s[0][1], s[0][2], d, 2},
                       {(void*)p[1], n[1][0], n[1][1], n[1][2], s[1][0], s[1][1], s[1][2], d, 2}};
    std::printf("%d\n", attn::apart(r[0], r[1]) + 2 * attn::apart(r[1], r[0]));
  }
}
"""


@pytest.fixture(scope="module")
def apart(tmp_path_factory):
    """apart(d, pairs): of each pair of (first element, sizes, strides), whether its sets are told to be apart."""
    t = tmp_path_factory.mktemp("apart")
    (t / "apart.cpp").write_text(PROGRAM)
    r = subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-I", CSRC, str(t / "apart.cpp"), "-o", str(t / "apart")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(d, pairs):
        text = "".join(f"{d} " + " ".join(str(v) for first, n, s in pair for v in (0x1000000 + 2 * first, *n, *s)) + "\n" for pair in pairs)
        out = subprocess.run([str(t / "apart")], input=text, capture_output=True, text=True, timeout=60)
        got = [int(v) for v in out.stdout.split()]
        assert out.returncode == 0 and len(got) == len(pairs) and set(got) <= {0, 3}  # the same either way round
        return [v == 3 for v in got]
    return run


def _elements(d, first, n, s):
    return {first + b * s[0] + h * s[1] + t * s[2] + i for b in range(n[0]) for h in range(n[1]) for t in range(n[2]) for i in range(d)}


# Axes of a packed array, slowest first: b batches, t tokens, h heads of one kind, k kinds (Q, K, V), j heads of all kinds.
ORDERS = ["btj", "bjt", "tbj", "jbt", "bthk", "bhtk", "tbkh", "kbth", "bkht", "bhkt", "hbtk", "tkbh"]


def _slices(order, B, N, H, Hkv, d):
    """(first, sizes, strides) of Q [B, H, N, d], K and V of a packed array; with kinds as an axis all have H heads."""
    size = {"b": B, "t": N, "h": H, "k": 3, "j": H + 2 * Hkv}
    stride, below = {}, d
    for a in reversed(order):
        stride[a], below = below, below * size[a]
    heads = "j" if "j" in order else "h"
    starts = [0, H * stride["j"], (H + Hkv) * stride["j"]] if heads == "j" else [k * stride["k"] for k in range(3)]
    counts = [H, Hkv, Hkv] if heads == "j" else [H] * 3
    return [(f, (B, c, N), (stride["b"], stride[heads], stride["t"])) for f, c in zip(starts, counts)]


@pytest.mark.parametrize("order", ORDERS)
def test_slices_of_packed_arrays_are_apart(apart, order):
    for B, N, H, Hkv, d in [(1, 1, 1, 1, 8), (2, 5, 3, 1, 8), (3, 1, 4, 2, 16), (1, 7, 2, 2, 8), (4, 3, 1, 1, 8), (2, 6, 6, 3, 16)]:
        q, k, v = _slices(order, B, N, H, Hkv, d)
        assert apart(d, [(q, k), (q, v), (k, v)]) == [True] * 3
        # Itself, and moved by a piece of 16 bytes into its neighbour, it is not.
        assert not any(apart(d, [(q, q), (q, (k[0] - 8, *k[1:])), (k, (v[0] - 8, *v[1:]))]))


def test_large_packed_arrays_are_apart(apart):
    for order in ORDERS:
        q, k, v = _slices(order, 16, 100003, 64, 8, 128)
        assert apart(128, [(q, k), (q, v), (k, v)]) == [True] * 3
        assert not any(apart(128, [(q, q), (q, (k[0] - 8, *k[1:]))]))


def test_what_is_told_apart_is(apart):
    """Any sizes and strides: never apart with an element in common; and few that are apart are not told so."""
    rnd, d, pairs, truth = random.Random(5), 8, [], []
    for _ in range(4000):
        strides = [8 * rnd.choice((0, 1, 2, 3, 4, 6, 8, 12, 16, 24, 40)) for _ in range(3)]
        sets = []
        for _ in range(2):
            n = tuple(rnd.randint(1, 4) for _ in range(3))
            s = tuple(strides if rnd.random() < 0.7 else [8 * rnd.randint(0, 30) for _ in range(3)])
            sets.append((8 * rnd.randint(0, 40), n, s))
        pairs.append(tuple(sets))
        truth.append(not (_elements(d, *sets[0]) & _elements(d, *sets[1])))
    got = apart(d, pairs)
    assert got == truth


P = 0x10000000


def _rows(first, strides):
    return pkg._Rows(P + 2 * first, *strides)


@pytest.mark.parametrize("order", ORDERS)
def test_overlapping_outputs_of_these_orders_are_refused(order):
    libbuild.build()
    lib = pkg.load_library()
    B, N, H, Hkv, d = 2, 5, 4, 4, 64
    q, k, v = _slices(order, B, N, H, Hkv, d)

    def call(qo, ko):
        return lib.attn_rope(_rows(q[0], q[2]), _rows(k[0], k[2]), _rows(qo[0], qo[2]), _rows(ko[0], ko[2]), None, 0, 0x40000000,
                             64, 0, 1.0, B, H, Hkv, N, d, 0, None)
    for qo, ko in [(k, k), (q, q), (k, q), ((q[0] + 8, *q[1:]), k), (q, (k[0] - 8, *k[1:])), (v, v), (v, (v[0] + 8, *v[1:]))]:
        assert call(qo, ko) == pkg.ATTN_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("module", [True, False])
@pytest.mark.parametrize("order", ORDERS)
def test_rotation_in_place_in_any_order(order, module, monkeypatch):
    if not module:
        monkeypatch.setattr(pkg, "_fast", False)
    B, N, H, Hkv, d = 2, 37, 4, 4, 64
    size = {"b": B, "t": N, "h": H, "k": 3, "j": H + 2 * Hkv}
    total = int(np.prod([size[a] for a in order])) * d
    x = torch.randn(total, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    before = x.clone()

    def rows(of, slc):
        first, (b, h, n), s = slc
        return torch.as_strided(of, (b, h, n, d), (*s, 1), first)
    slices = _slices(order, B, N, H, Hkv, d)
    freqs, _ = pkg.attn_rope_freqs(d)
    q, k, v = (rows(x, s) for s in slices)
    want = pkg.attn_rope(*(rows(before, s).contiguous() for s in slices[:2]), freqs)
    pkg.attn_rope(q, k, freqs, Q_out=q, K_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, rows(before, slices[2]))
    # K's turned rows over V's: the last kind's place is an output between the others.
    pkg.attn_rope(k, None, freqs, Q_out=v)
    assert torch.equal(v, pkg.attn_rope(want[1], None, freqs)[0]) and torch.equal(q, want[0])
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK
