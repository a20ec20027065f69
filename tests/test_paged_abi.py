"""Refusals of the paged cache's calls: by the library before it touches the GPU
(no GPU needed), and by the Python layer."""

import ctypes

import pytest
import torch

import exact_attention_95_gb300 as pkg
from exact_attention_95_gb300 import build as libbuild

BAD, NO = pkg.ATTN_ERR_INVALID_ARG, pkg.ATTN_ERR_UNSUPPORTED
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkg.load_library()


def at(k):
    return P(0x100000 * (k + 1))  # fake, aligned, far apart; never dereferenced on these paths


def _tables(lib, **kw):
    a = dict(cached=at(0), added=at(1), free=at(2), F=10, table=at(3), width=4, page=16, lens=at(4), cu=at(5),
             slots=at(6), pos=at(7), taken=at(8), R=3, T=5)
    a.update(kw)
    return lib.attn_kv_tables(a["cached"], a["added"], a["free"], a["F"], a["table"], a["width"], a["page"], a["lens"],
                              a["cu"], a["slots"], a["pos"], a["taken"], a["R"], a["T"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(cached=None), BAD), (dict(added=None), BAD), (dict(table=None), BAD), (dict(lens=None), BAD),
    (dict(cu=None), BAD), (dict(taken=None), BAD), (dict(free=None), BAD), (dict(slots=None), BAD),
    (dict(pos=None), BAD), (dict(R=0), BAD), (dict(T=-1), BAD), (dict(F=-1), BAD), (dict(width=0), BAD),
    (dict(page=0), BAD), (dict(page=24), NO), (dict(page=8), NO), (dict(page=256), NO), (dict(width=2 ** 27), NO),
    (dict(T=2 ** 31 - 1), NO), (dict(F=2 ** 31 - 1, free=P(0x7000000000)), NO),
    (dict(cached=P(0x100002)), BAD), (dict(slots=P(0x700004)), BAD), (dict(taken=P(0x900001)), BAD),
    # Outputs over inputs.
    (dict(lens=at(0)), BAD), (dict(cu=P(0x100000 - 4)), BAD), (dict(pos=P(0x300000 + 36)), BAD), (dict(table=at(2)), BAD),
], ids=str)
def test_tables_argument_errors(lib, kw, want):
    assert _tables(lib, **kw) == want


def _append(lib, **kw):
    a = dict(K=at(0), ks=1024, V=at(1), vs=1024, slots=at(2), kp=at(3), ksc=at(4), vp=at(5), vsc=at(6), T=5, Hkv=8,
             d=128, pages=10, page=64)
    a.update(kw)
    return lib.attn_kv_append_fp8(a["K"], a["ks"], a["V"], a["vs"], a["slots"], a["kp"], a["ksc"], a["vp"], a["vsc"],
                                  a["T"], a["Hkv"], a["d"], a["pages"], a["page"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(K=None), BAD), (dict(V=None), BAD), (dict(slots=None), BAD), (dict(kp=None), BAD), (dict(vsc=None), BAD),
    (dict(K=P(0x100008)), BAD), (dict(vp=P(0x600008)), BAD), (dict(ksc=P(0x500002)), BAD), (dict(slots=P(0x300004)), BAD),
    (dict(ks=1016), BAD), (dict(vs=1028), BAD), (dict(T=-1), BAD), (dict(Hkv=0), BAD), (dict(pages=0), BAD),
    (dict(page=-1), BAD), (dict(d=96), NO), (dict(page=48), NO), (dict(Hkv=32768, ks=2 ** 23, vs=2 ** 23), NO),
    (dict(pages=2 ** 29), NO), (dict(T=0, K=None, V=None, slots=None), pkg.ATTN_OK),
], ids=str)
def test_append_argument_errors(lib, kw, want):
    assert _append(lib, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(vp=at(3)), dict(vsc=at(4)), dict(ksc=P(0x400000 + 10 * 8 * 64 * 128 - 4)), dict(slots=at(6)), dict(K=at(5)),
    dict(V=P(0x400000 - 2 * (4 * 1024 + 1024) + 16)), dict(vsc=P(0x500000 + 10 * 8 * 4 - 4)),
], ids=str)
def test_append_refuses_arrays_that_overlap_what_it_updates(lib, kw):
    assert _append(lib, **kw) == BAD


def _fwd(lib, **kw):
    a = dict(Q=at(0), qs=4096, kp=at(1), ks=at(2), vp=at(3), vs=at(4), table=at(5), cu=at(6), lens=at(7), O=at(8),
             L=at(9), R=3, T=5, Hq=32, Hkv=8, d=128, pages=10, page=64, width=4, scale=0.1, causal=1, out=0, ws=at(10),
             wsb=1 << 40)
    a.update(kw)
    return lib.attn_fwd_paged_fp8(a["Q"], a["qs"], a["kp"], a["ks"], a["vp"], a["vs"], a["table"], a["cu"], a["lens"],
                                  a["O"], a["L"], a["R"], a["T"], a["Hq"], a["Hkv"], a["d"], a["pages"], a["page"],
                                  a["width"], a["scale"], a["causal"], a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    *[({k: None}, BAD) for k in ("Q", "kp", "ks", "vp", "vs", "table", "cu", "lens", "O", "L", "ws")],
    (dict(Q=P(0x100008)), BAD), (dict(O=P(0x900008)), BAD), (dict(L=P(0xa00002)), BAD), (dict(ws=P(0xb00080)), BAD),
    (dict(table=P(0x600002)), BAD), (dict(qs=4088), BAD), (dict(qs=4100), BAD), (dict(R=0), BAD), (dict(T=-1), BAD),
    (dict(Hq=30), BAD), (dict(Hq=0), BAD), (dict(width=0), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(causal=2), BAD), (dict(out=3), BAD),
    (dict(d=256, qs=8192), NO), (dict(page=100), NO), (dict(R=16385), NO), (dict(T=2 ** 26), NO),
    (dict(width=2 ** 25, page=64), NO), (dict(T=0, Q=None, O=None, L=None, ws=None), pkg.ATTN_OK),
], ids=str)
def test_attention_argument_errors(lib, kw, want):
    assert _fwd(lib, **kw) == want


def test_workspace_size(lib):
    size = pkg.attn_fwd_paged_workspace_size
    assert size(4, 4, 32, 8, 128) > 0
    # A decoding step needs no room for tiles of many rows.
    assert size(4, 4, 32, 8, 128) < size(4, 5, 32, 8, 128) and size(4, 4, 32, 2, 128) == size(4, 5, 32, 2, 128)
    for bad in ((0, 4, 32, 8, 128), (4, 0, 32, 8, 128), (4, 4, 30, 8, 128), (4, 4, 32, 8, 96), (4, 4, 0, 8, 128)):
        assert size(*bad) == 0


def test_binding_rejects_host_tensors():
    i = torch.zeros(3, dtype=torch.int32)
    t = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        pkg.attn_kv_tables(i, i, i, t, 16, 3)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pages, scale = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.ones(4, 2)
    with pytest.raises(TypeError):
        pkg.attn_kv_append_fp8(x, x, torch.zeros(3, dtype=torch.int64), pages, scale, pages, scale)
    with pytest.raises(TypeError):
        pkg.attn_fwd_paged_fp8(x, pages, scale, pages, scale, t, i, i)
    with pytest.raises(KeyError):
        pkg.attn_fwd_paged_fp8(x, pages, scale, pages, scale, t, i, i, out_dtype=torch.float16)


@pytest.mark.gpu
def test_binding_rejects_bad_tensors_on_gpu():
    dev = "cuda"
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=dev)
    table = torch.zeros(3, 2, dtype=torch.int32, device=dev)
    ok = dict(cached=i32(3), added=i32(3), free_pages=i32(4), block_table=table, page_size=16, T=3)
    pkg.attn_kv_tables(**ok)
    for exc, kw in [(ValueError, dict(added=i32(4))), (TypeError, dict(added=i32(3).long())),
                    (ValueError, dict(block_table=table.t().contiguous().t())), (TypeError, dict(block_table=i32(6))),
                    (ValueError, dict(kv_lens=i32(4))), (TypeError, dict(slots=i32(3))),
                    (ValueError, dict(slots=torch.zeros(6, dtype=torch.int64, device=dev)[::2])),
                    (TypeError, dict(free_pages=torch.zeros(4, dtype=torch.int32))),
                    (pkg.AttnError, dict(page_size=20)), (pkg.AttnError, dict(kv_lens=ok["cached"]))]:
        with pytest.raises(exc):
            pkg.attn_kv_tables(**{**ok, **kw})
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=dev)
    kv = x[:, :2]
    pages, scale = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=dev), torch.ones(4, 2, device=dev)
    slots = torch.full((3,), -1, dtype=torch.int64, device=dev)
    pkg.attn_kv_append_fp8(kv, kv, slots, pages, scale, pages.clone(), scale.clone())
    for exc, args in [(TypeError, (kv.float(), kv, slots, pages, scale, pages, scale)),
                      (ValueError, (x, kv, slots, pages, scale, pages, scale)),
                      (ValueError, (kv, kv[:2], slots, pages, scale, pages, scale)),
                      (ValueError, (kv, x[:, ::2], slots, pages, scale, pages, scale)),
                      (ValueError, (kv, kv, slots[:2], pages, scale, pages, scale)),
                      (ValueError, (kv, kv, slots, pages, scale, pages[:3], scale)),
                      (TypeError, (kv, kv, slots, pages, scale.double(), pages, scale)),
                      (pkg.AttnError, (kv, kv, slots, pages[:, :, :8].contiguous(), scale, pages[:, :, :8].contiguous(),
                                       scale))]:
        with pytest.raises(exc):
            pkg.attn_kv_append_fp8(*args)
    cu, lens = i32(4), i32(3)
    good = dict(Q=x, k_pages=pages, k_scale=scale, v_pages=pages, v_scale=scale, block_table=table, cu_q=cu, kv_lens=lens)
    pkg.attn_fwd_paged_fp8(**good)
    small = torch.empty(16, dtype=torch.uint8, device=dev)
    for exc, kw in [(ValueError, dict(cu_q=lens)), (TypeError, dict(kv_lens=lens.long())),
                    (ValueError, dict(Q=x[:, :, :32])), (ValueError, dict(workspace=small)),
                    (ValueError, dict(O=torch.empty(3, 4, 32, dtype=torch.bfloat16, device=dev))),
                    (TypeError, dict(O=torch.empty(3, 4, 64, device=dev))), (TypeError, dict(LSE=x)),
                    (pkg.AttnError, dict(Q=x[:, :3].contiguous())), (pkg.AttnError, dict(scale=0.0)),
                    (pkg.AttnError, dict(block_table=table[:0], cu_q=cu[:1], kv_lens=lens[:0]))]:
        with pytest.raises(exc):
            pkg.attn_fwd_paged_fp8(**{**good, **kw})
    # Nothing to do is no error.
    O, L = pkg.attn_fwd_paged_fp8(**{**good, "Q": x[:0]})
    assert O.shape == (0, 4, 64) and L.shape == (0, 4)


@pytest.mark.gpu
def test_a_named_stream_and_given_outputs():
    """The calls on a stream that is not current, and with every output given, give what they give without."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(5)
    cached, added = (torch.randint(0, 40, (5,), generator=g, device=dev).int() for _ in range(2))
    free = torch.arange(20, 60, dtype=torch.int32, device=dev)
    table = torch.arange(20, dtype=torch.int32, device=dev).reshape(5, 4).repeat(1, 2).contiguous()
    T = 210
    k, v, q = (torch.randn(T, h, 64, generator=g, device=dev).bfloat16() for h in (2, 2, 6))

    def step(stream, given):
        tb = table.clone()
        c = [torch.zeros(60, 2, 16, 64, dtype=torch.uint8, device=dev), torch.ones(60, 2, device=dev)]
        c += [c[0].clone(), c[1].clone()]
        outs = {}
        if given:
            i32 = lambda n: torch.empty(n, dtype=torch.int32, device=dev)
            outs = dict(kv_lens=i32(5), cu_tokens=i32(6), slots=torch.empty(T, dtype=torch.int64, device=dev),
                        positions=i32(T), taken=i32(2))
        torch.cuda.synchronize()
        lens, cu, slots, pos, taken = pkg.attn_kv_tables(cached, added, free, tb, 16, T, stream=stream, **outs)
        pkg.attn_kv_append_fp8(k, v, slots, *c, stream=stream)
        more = dict(O=torch.empty_like(q), LSE=torch.empty(T, 6, device=dev)) if given else {}
        torch.cuda.synchronize()
        O, L = pkg.attn_fwd_paged_fp8(q, *c, tb, cu, lens, causal=True, stream=stream, **more)
        torch.cuda.synchronize()
        n = int(cu[-1])
        return [tb, lens, cu, slots, pos, taken, *c, O[:n], L[:n]]

    want = step(None, False)
    for stream, given in ((torch.cuda.Stream(), False), (None, True), (torch.cuda.Stream(), True)):
        assert all(torch.equal(a, b) for a, b in zip(want, step(stream, given)))
    assert pkg.attn_last_device_status() == pkg.ATTN_OK
