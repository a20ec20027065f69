"""The paged cache's kernels in the debug variant of the library: every check of a
copy's coordinate and of a store's index passes, and the outputs are the
release library's."""

import os
import subprocess
import sys

import pytest

from exact_attention_95_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Steps of a server in every kernel: (new tokens of the requests, heads, kv heads, d, page, columns of the table
# behind what the requests need, requests refused for want of pages).
SCRIPT = r"""
import sys
import torch
import exact_attention_95_gb300 as pkg
assert pkg.LIB_PATH.endswith("_debug.so") == (sys.argv[1] == "debug")
CASES = [
    ([[70, 0, 130], [1, 1, 1]], 8, 2, 128, 16, 0, False),      # clusters
    ([[70, 0, 130], [1, 1, 1]], 8, 2, 64, 128, 100, False),    # ranges, 8 rows
    ([[500, 40], [5, 3], [1, 6]], 8, 2, 128, 32, 0, False),    # 16 rows
    ([[500, 40], [5, 3], [40, 9]], 4, 2, 64, 64, 0, True),     # 16 and 256 rows
    ([[300], [200]], 2, 2, 128, 128, 3, False),                # 256 rows
    ([[9] * 70, [1] * 70, [2] * 70], 4, 1, 64, 16, 0, True),   # more than 32 requests
    ([[9] * 300, [1] * 300], 32, 2, 128, 16, 0, False),        # 16 heads a kv head
]
out = []
for n, (steps, Hq, Hkv, d, page, extra, short) in enumerate(CASES):
    g = torch.Generator(device="cuda").manual_seed(n)
    R = len(steps[0])
    total = [sum(s[r] for s in steps) for r in range(R)]
    need = [-(-x // page) for x in total]
    num_pages = sum(need)
    free = torch.randperm(num_pages, generator=g, device="cuda").int()
    if short:
        free = free[:num_pages - 2].contiguous()
    table = torch.zeros(R, max(need) + extra, dtype=torch.int32, device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    cache = [x for _ in range(2) for x in (torch.zeros(num_pages, Hkv, page, d, dtype=torch.uint8, device="cuda"),
                                           torch.ones(num_pages, Hkv, device="cuda"))]
    for s in steps:
        T = sum(s) + 3
        q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
        added = torch.tensor(s, dtype=torch.int32, device="cuda")
        lens, cu, slots, pos, taken = pkg.attn_kv_tables(lens, added, free, table, page, T)
        free = free[int(taken[0]):]
        pkg.attn_kv_append_fp8(k, v, slots, *cache)
        for dtype in (torch.bfloat16, torch.float32):
            O, L = (torch.zeros(T, Hq, d, dtype=dtype, device="cuda"), torch.zeros(T, Hq, device="cuda"))
            pkg.attn_fwd_paged_fp8(q, *cache, table, cu, lens, causal=True, out_dtype=dtype, O=O, LSE=L)
            out += [O.cpu(), L.cpu()]
        out += [x.cpu() for x in (lens, cu, slots, pos, taken)]
    out += [x.cpu() for x in (table, *cache)]
torch.cuda.synchronize()
st = pkg.attn_last_device_status()
assert st == pkg.ATTN_OK, pkg.attn_status_string(st)
torch.save(out, sys.argv[2])
"""


@pytest.mark.gpu
def test_the_debug_variant_runs_the_paged_kernels_clean_and_as_the_release_does(tmp_path):
    import torch
    libbuild.build(debug=True)
    got = {}
    for kind in ("debug", "release"):
        path = str(tmp_path / kind)
        env = dict(os.environ, ATTN_DEBUG="1" if kind == "debug" else "0", PYTHONPATH=ROOT)
        r = subprocess.run([sys.executable, "-c", SCRIPT, kind, path], env=env, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr
        got[kind] = torch.load(path)
    assert len(got["debug"]) == len(got["release"]) > 0
    for a, b in zip(got["debug"], got["release"]):
        assert a.dtype == b.dtype and torch.equal(a, b)
    assert sum(int(x[1]) > 0 for x in got["release"] if x.dtype == torch.int32 and x.numel() == 2) > 0  # refusals among them
