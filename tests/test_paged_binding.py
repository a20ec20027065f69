"""The extension module of the paged cache's calls: nothing else depends on it, and
without it the calls give the same."""

import os
import subprocess
import sys

import pytest
import torch

import exact_attention_95_gb300 as pkg
from exact_attention_95_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys, warnings
import torch
import exact_attention_95_gb300 as pkg
from exact_attention_95_gb300 import build
sys.modules[pkg.__name__ + "._binding"] = None  # no import of it succeeds
build.binding_path = lambda: "%s"
assert pkg.attn_bwd_workspace_size(2, 4, 2, 100, 64) > 0 and pkg.attn_fwd_paged_workspace_size(4, 4, 32, 8, 128) > 0
assert pkg.attn_status_string(0) == "ATTN_OK"
x = torch.zeros(3, dtype=torch.int32)
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    for _ in range(2):  # (the second call does not warn again)
        try:
            pkg.attn_kv_tables(x, x, x, torch.zeros(3, 2, dtype=torch.int32), 16, 3)
        except TypeError as e:
            assert "cached must be a CUDA tensor" in str(e)
        else:
            raise AssertionError("a host tensor was taken")
assert [x.category for x in w] == [RuntimeWarning], w
print("without it")
"""


@pytest.mark.parametrize("what", ["missing", "not a module"])
def test_the_library_loads_without_the_module(what, tmp_path):
    libbuild.build()
    path = tmp_path / "none.so"
    if what == "not a module":
        path.write_bytes(b"not a shared object")
    r = subprocess.run([sys.executable, "-c", WITHOUT % path], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "without it" in r.stdout, r.stderr[-2000:]


def test_the_modules_name_has_the_versions_it_is_built_for(monkeypatch):
    import sysconfig
    path = libbuild.binding_path()
    assert torch.__version__ in path and sysconfig.get_config_var("SOABI") in path
    assert os.path.exists(libbuild.build_binding())
    monkeypatch.setattr(torch, "__version__", "1.2.3")
    assert libbuild.binding_path() != path and not os.path.exists(libbuild.binding_path())


def test_the_library_is_built_where_the_module_cannot_be(monkeypatch, tmp_path):
    """And a module of older sources is not left for it to be called by."""
    def fail(force=False):
        raise RuntimeError("Python.h: no such file")

    libbuild.build()
    old = tmp_path / "old.so"
    old.write_bytes(b"a module of older sources")
    monkeypatch.setattr(libbuild, "build_binding", fail)
    monkeypatch.setattr(libbuild, "binding_path", lambda: str(old))
    for _ in range(2):
        with pytest.warns(RuntimeWarning, match="Python.h"):
            assert os.path.exists(libbuild.build())
        assert not old.exists()


def test_the_module_is_the_one_that_is_used():
    libbuild.build()
    assert pkg._bound() and pkg._bound().__file__ == libbuild.binding_path()


def _step(R, T, d):
    """Tables, append and attention of a step; every output and every updated array."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(R + T)
    added = torch.full((R,), T // R, dtype=torch.int32, device=dev)
    cached = torch.randint(0, 50, (R,), generator=g, device=dev).int()
    free = torch.arange(8 * R, 16 * R, dtype=torch.int32, device=dev)
    table = torch.arange(8 * R, dtype=torch.int32, device=dev).reshape(R, 8).contiguous()
    q, k, v = (torch.randn(T, h, d, generator=g, device=dev).bfloat16() for h in (6, 2, 2))
    cache = [torch.zeros(16 * R, 2, 16, d, dtype=torch.uint8, device=dev), torch.ones(16 * R, 2, device=dev)]
    cache += [c.clone() for c in cache]
    lens, cu, slots, pos, taken = pkg.attn_kv_tables(cached, added, free, table, 16, T)
    pkg.attn_kv_append_fp8(k, v, slots, *cache)
    O, L = pkg.attn_fwd_paged_fp8(q, *cache, table, cu, lens, causal=True)
    O32, L32 = pkg.attn_fwd_paged_fp8(q, *cache, table, cu, lens, 0.1, False, torch.float32)
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK
    return [table, lens, cu, slots, pos, taken, *cache, O, L, O32, L32]


@pytest.mark.gpu
@pytest.mark.parametrize("R,T,d", [(3, 3, 64), (4, 60, 128)])
def test_the_calls_give_the_same_without_the_module(R, T, d, monkeypatch):
    want = _step(R, T, d)
    assert pkg._bound()
    monkeypatch.setattr(pkg, "_fast", False)
    for a, b in zip(want, _step(R, T, d)):
        assert a.dtype == b.dtype and torch.equal(a, b)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    x, i = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    pages, one = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda"), torch.ones(4, 2, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        pkg.attn_fwd_paged_fp8(x, pages, one, pages, one, i[:, None].repeat(1, 2).contiguous(), torch.zeros_like(i[:1]).repeat(4),
                               i, workspace=small)


@pytest.mark.gpu
@pytest.mark.parametrize("module", [True, False])
def test_an_allocation_that_fails_raises_as_torch_raises_it(module, monkeypatch):
    """Eight gigabytes and more of outputs where the process may have three (nothing is allocated)."""
    if not module:
        monkeypatch.setattr(pkg, "_fast", False)
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.01)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            pkg.attn_kv_tables(i, i, i, table, 16, 10 ** 9)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    pkg.attn_kv_tables(i, i, i, table, 16, 3)
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("module", [True, False])
def test_what_outputs_share(module, monkeypatch):
    """Keeping, saving or resizing an output takes no other along, but for the small ones
    of the tables (a few bytes a request) among one another."""
    if not module:
        monkeypatch.setattr(pkg, "_fast", False)
    R = 4
    table, lens, cu, slots, pos, taken, *rest = _step(R, 60, 64)
    own = [slots, pos, *rest]
    for t in own:
        assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * t.element_size()
    for t in (lens, cu, taken):
        assert t.untyped_storage().nbytes() <= 4 * (2 * R + 3)
    at = [t.untyped_storage().data_ptr() for t in own]
    assert len(set(at)) == len(at) and not {t.untyped_storage().data_ptr() for t in (lens, cu, taken)} & set(at)
