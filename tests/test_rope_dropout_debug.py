"""Rotary positions, the append with them, and attention with dropout in the debug variant of the
library: every check of a copy's coordinate and of a store's index passes, and the outputs are
the release library's (but for dQ, whose sums have no fixed order)."""

import os
import subprocess
import sys

import pytest

from exact_attention_95_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys
import torch
import exact_attention_95_gb300 as pkg
assert pkg.LIB_PATH.endswith("_debug.so") == (sys.argv[1] == "debug")
out, loose = [], []
g = torch.Generator(device="cuda").manual_seed(1)
rng = torch.tensor([5, 6], device="cuda")
for B, Hq, Hkv, N, d, rot, inter in [(1, 4, 2, 300, 128, 128, False), (2, 2, 2, 257, 64, 32, True), (1, 8, 2, 30, 128, 48, False),
                                     (3, 2, 1, 640, 64, 64, False), (1, 1, 1, 1, 128, 128, True), (1, 2, 2, 128, 64, 64, True)]:
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g, device="cuda").bfloat16()
    q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    freqs, _ = pkg.attn_rope_freqs(rot)
    Q, K = pkg.attn_rope(q, k, freqs, None, inter)
    V, dO = v.contiguous(), torch.randn(B, Hq, N, d, generator=g, device="cuda").bfloat16()
    for p in (0.1, 0.7):
        O, L = pkg.attn_fwd_dropout(Q, K, V, p, rng, None, N % 2 == 0)
        dQ, dK, dV = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, p, rng, None, N % 2 == 0)
        out += [O, L, dK, dV]
        loose.append(dQ)
    out += [Q, K, *pkg.attn_rope_bwd(Q.float(), K.float(), freqs, None, inter)]
for lens, page, Hq, Hkv, d in [([1, 1, 5], 16, 4, 2, 64), ([300, 20, 9], 64, 6, 3, 128), ([9] * 200, 32, 8, 8, 64)]:
    T, R = sum(lens) + 2, len(lens)
    free = torch.randperm(2 * R + T // page + 9, generator=g, device="cuda").int()
    table = torch.zeros(R, 20, dtype=torch.int32, device="cuda")
    cache = [c for _ in range(2) for c in (torch.zeros(len(free), Hkv, page, d, dtype=torch.uint8, device="cuda"),
                                           torch.ones(len(free), Hkv, device="cuda"))]
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device="cuda").bfloat16()
    added = torch.tensor(lens, dtype=torch.int32, device="cuda")
    have = torch.full_like(added, 3)
    table[:, 0] = free[:R]
    _, _, slots, pos, _ = pkg.attn_kv_tables(have, added, free[R:].contiguous(), table, page, T)
    for inter in (False, True):
        freqs, _ = pkg.attn_rope_freqs(d // 2)
        out.append(pkg.attn_kv_append_rope_fp8(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos, slots, freqs, *cache, inter))
        out += [c.clone() for c in cache]
torch.cuda.synchronize()
st = pkg.attn_last_device_status()
assert st == pkg.ATTN_OK, pkg.attn_status_string(st)
torch.save([[t.cpu() for t in out], [t.cpu() for t in loose]], sys.argv[2])
"""


@pytest.mark.gpu
def test_the_debug_variant_runs_them_clean_and_as_the_release_does(tmp_path):
    import torch
    libbuild.build(debug=True)
    got = {}
    for kind in ("debug", "release"):
        path = str(tmp_path / kind)
        env = dict(os.environ, ATTN_DEBUG="1" if kind == "debug" else "0", PYTHONPATH=ROOT)
        r = subprocess.run([sys.executable, "-c", SCRIPT, kind, path], env=env, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr
        got[kind] = torch.load(path)
    assert len(got["debug"][0]) == len(got["release"][0]) > 0
    for a, b in zip(got["debug"][0], got["release"][0]):
        assert a.dtype == b.dtype and torch.equal(a, b)
    for a, b in zip(got["debug"][1], got["release"][1]):
        # fp32 sums in another order, then bf16: a step of the largest element at most.
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max() + 1e-6
