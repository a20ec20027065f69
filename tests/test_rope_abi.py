"""Rotary positions without a GPU: the plain implementation on known values, the
frequencies against their formulas, and refusals by the library and the Python layer."""

import ctypes
import math

import numpy as np
import pytest
import torch

import exact_attention_95_gb300 as pkg
from exact_attention_95_gb300 import build as libbuild

import positions as pos64

BAD, NO = pkg.ATTN_ERR_INVALID_ARG, pkg.ATTN_ERR_UNSUPPORTED
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return pkg.load_library()


def at(k):
    return 0x10000000 * (k + 1)  # fake, aligned, far apart; never dereferenced on these paths


# ------------------------------------------------------------------ plain implementation
def test_plain_rotation_on_known_values():
    quarter = [2 ** 62] * 2  # a quarter turn a position
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    y, size = pos64.rotate(x, [1], quarter, False, 1.0)
    assert np.allclose(y, [[[-3.0, -4.0, 1.0, 2.0, 5.0]]]) and np.allclose(size, [[[4.0, 6.0, 4.0, 6.0, 0.0]]])
    y, _ = pos64.rotate(x, [1], quarter, True, 2.0)
    assert np.allclose(y, [[[-4.0, 2.0, -8.0, 6.0, 5.0]]])
    assert np.array_equal(pos64.rotate(x, [-1], quarter, True, 2.0)[0], x)
    # Four quarters are none, however far; the gradient's turn is the way back.
    assert np.allclose(pos64.rotate(x, [2 ** 31 - 4], quarter, False, 1.0)[0], x)
    back = pos64.rotate(pos64.rotate(x, [77], [2 ** 60, 12345], False, 1.0)[0], [77], [2 ** 60, 12345], False, 1.0, -1.0)
    assert np.allclose(back[0], x)


# ------------------------------------------------------------------ frequencies
@pytest.mark.parametrize("rot", [2, 16, 64, 128, 1024])
@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
    dict(scaling="parts", factor=16.0, original_len=4096), dict(scaling="parts", factor=2.5, original_len=300, low=2, high=9),
    dict(scaling="parts", factor=1.0, original_len=2048),
], ids=str)
def test_frequencies_are_those_of_their_formulas(lib, rot, kw):
    if rot == 2 and kw.get("scaling") == "base":
        with pytest.raises(pkg.AttnError, match="INVALID_ARG"):
            pkg.attn_rope_freqs(rot, device="cpu", **kw)
        return
    freqs, amplitude = pkg.attn_rope_freqs(rot, device="cpu", **kw)
    want, a = pos64.frequencies(rot, **kw)
    assert freqs.dtype == torch.int64 and freqs.shape == (rot // 2,) and amplitude == pytest.approx(a, rel=1e-14)
    # A few operations in 64 bits (2^-53 each), and a power whose exponent's rounding its logarithm magnifies (below 32 of them).
    assert np.abs(freqs.numpy() / 2.0 ** 64 / want - 1).max() < 64 * 2.0 ** -53 + 2.0 ** -64 / want.min()
    assert (freqs > 0).all()


def test_scaled_frequencies_end_where_they_have_to(lib):
    plain, _ = pkg.attn_rope_freqs(128, device="cpu")
    for kw in (dict(scaling="base"), dict(scaling="parts", original_len=4096)):
        f, _ = pkg.attn_rope_freqs(128, factor=8.0, device="cpu", **kw)
        assert abs(int(f[0]) / int(plain[0]) - 1) < 1e-12 and abs(8 * int(f[-1]) / int(plain[-1]) - 1) < 1e-12


@pytest.mark.parametrize("kw,want", [
    (dict(rot=0), BAD), (dict(rot=-2), BAD), (dict(rot=3), NO), (dict(rot=1026), NO), (dict(base=1.0), BAD),
    (dict(base=float("inf")), BAD), (dict(base=float("nan")), BAD), (dict(scaling=4), BAD), (dict(scaling=-1), BAD),
    (dict(scaling=1, factor=0.5), BAD), (dict(scaling=2, factor=float("nan")), BAD), (dict(scaling=3, original=0.0), BAD),
    (dict(scaling=3, low=32.0), BAD), (dict(scaling=3, low=-1.0), BAD), (dict(scaling=3, high=float("inf")), BAD),
    (dict(freqs=None), BAD), (dict(amp=None), BAD), (dict(factor=0.0, original=-1.0, low=9.0, high=1.0), pkg.ATTN_OK),
], ids=str)
def test_frequency_refusals(lib, kw, want):
    out, amp = (ctypes.c_uint64 * 512)(), ctypes.c_double()
    a = dict(freqs=ctypes.addressof(out), amp=ctypes.addressof(amp), rot=64, base=1e4, scaling=0, factor=2.0,
             original=4096.0, low=1.0, high=32.0)
    a.update(kw)
    assert lib.attn_rope_freqs(a["freqs"], a["amp"], a["rot"], a["base"], a["scaling"], a["factor"], a["original"],
                               a["low"], a["high"]) == want


def test_python_frequency_refusals(lib):
    with pytest.raises(ValueError, match="scaling"):
        pkg.attn_rope_freqs(64, scaling="other", device="cpu")
    with pytest.raises(pkg.AttnError, match="UNSUPPORTED"):
        pkg.attn_rope_freqs(63, device="cpu")


# ------------------------------------------------------------------ refusals
def _rows(base, batch=0, head=0, token=0):
    return pkg._Rows(base, batch, head, token)


def _rope(lib, bwd=False, **kw):
    """Q, K as slices of a packed [2, 5, 6, 128] projection, outputs [2, H, 5, 128]."""
    a = dict(Q=_rows(at(0), 3840, 128, 768), K=_rows(at(0) + 2 * 512, 3840, 128, 768), Qo=_rows(at(1), 2560, 640, 128),
             Ko=_rows(at(2), 640, 640, 128), pos=at(3), pb=5, freqs=at(4), rot=128, inter=0, amp=1.0, B=2, Hq=4, Hkv=1,
             N=5, d=128, dtype=0)
    a.update(kw)
    f = lib.attn_rope_bwd if bwd else lib.attn_rope
    return f(a["Q"], a["K"], a["Qo"], a["Ko"], a["pos"], a["pb"], a["freqs"], a["rot"], a["inter"], a["amp"], a["B"],
             a["Hq"], a["Hkv"], a["N"], a["d"], a["dtype"], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(Q=None), BAD), (dict(Qo=None), BAD), (dict(K=None), BAD), (dict(Ko=None), BAD), (dict(freqs=None), BAD),
    (dict(Q=_rows(None, 3840, 128, 768)), BAD), (dict(Qo=_rows(at(1) + 8, 2560, 640, 128)), BAD),
    (dict(Q=_rows(at(0), 3840, 128, 772)), BAD), (dict(K=_rows(at(0), 3840, -128, 768), Hkv=2), BAD),
    (dict(pos=at(3) + 2), BAD), (dict(freqs=at(4) + 4), BAD), (dict(pb=-1), BAD), (dict(B=0), BAD), (dict(Hq=0), BAD),
    (dict(Hkv=0), BAD), (dict(N=-1), BAD), (dict(rot=0), BAD), (dict(rot=144), BAD), (dict(rot=24), NO), (dict(d=96, rot=96), NO),
    (dict(d=256), NO), (dict(inter=2), BAD), (dict(amp=0.0), BAD), (dict(amp=-1.0), BAD), (dict(amp=float("inf")), BAD),
    (dict(dtype=2), BAD), (dict(N=2 ** 30, B=4), NO), (dict(Hq=65535), NO), (dict(N=0), pkg.ATTN_OK),
    # Rows of an output that share elements.
    (dict(Qo=_rows(at(1), 2560, 640, 0)), BAD), (dict(Qo=_rows(at(1), 2560, 64, 128)), BAD),
    (dict(Ko=_rows(at(2), 0, 640, 128)), BAD),
    # Outputs over other arrays of the call.
    (dict(Qo=_rows(at(2), 2560, 640, 128)), BAD), (dict(Ko=_rows(at(1) + 256, 640, 640, 128)), BAD),
    (dict(Ko=_rows(at(0), 3840, 128, 768)), BAD),                   # K_out over Q's first head
    (dict(Qo=_rows(at(0) + 256, 3840, 128, 768)), BAD),             # one head on from Q
    (dict(Qo=_rows(at(0), 3840, 128, 640)), BAD), (dict(Qo=_rows(at(0), 2560, 640, 128)), BAD),
    (dict(K=_rows(at(5), 640, 640, 128), Ko=_rows(at(0) + 2 * 512 - 16, 3840, 128, 768)), BAD),  # a piece over Q's last head
    (dict(Qo=_rows(at(3) - 256, 2560, 640, 128)), BAD), (dict(Ko=_rows(at(4), 640, 640, 128)), BAD),
], ids=str)
def test_rope_refusals(lib, bwd, kw, want):
    assert _rope(lib, bwd, **kw) == want


def _append(lib, **kw):
    a = dict(Q=at(0), qs=768, K=at(0) + 2 * 512, ks=768, V=at(0) + 2 * 640, vs=768, pos=at(1), slots=at(2), freqs=at(3),
             rot=128, inter=0, amp=1.0, Qo=at(4), qos=512, kp=at(5), ksc=at(6), vp=at(7), vsc=at(8), T=5, Hq=4, Hkv=1,
             d=128, pages=10, page=64)
    a.update(kw)
    return lib.attn_kv_append_rope_fp8(a["Q"], a["qs"], a["K"], a["ks"], a["V"], a["vs"], a["pos"], a["slots"], a["freqs"],
                                       a["rot"], a["inter"], a["amp"], a["Qo"], a["qos"], a["kp"], a["ksc"], a["vp"],
                                       a["vsc"], a["T"], a["Hq"], a["Hkv"], a["d"], a["pages"], a["page"], None)


@pytest.mark.parametrize("kw,want", [
    *[({k: None}, BAD) for k in ("Q", "K", "V", "pos", "slots", "freqs", "Qo", "kp", "ksc", "vp", "vsc")],
    (dict(Q=at(0) + 8), BAD), (dict(Qo=at(4) + 8), BAD), (dict(pos=at(1) + 2), BAD), (dict(freqs=at(3) + 4), BAD),
    (dict(slots=at(2) + 4), BAD), (dict(qs=504), BAD), (dict(qs=772), BAD), (dict(qos=516), BAD), (dict(ks=120), BAD),
    (dict(T=-1), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(rot=0), BAD), (dict(rot=129), BAD), (dict(rot=40), NO),
    (dict(inter=-1), BAD), (dict(amp=float("nan")), BAD), (dict(d=96, rot=96), NO), (dict(page=24), NO), (dict(Hq=65536, qs=2 ** 23, qos=2 ** 23), NO),
    (dict(T=0, Q=None, K=None, V=None, pos=None, slots=None, freqs=None, Qo=None), pkg.ATTN_OK),
    # What is written over another array of the call.
    (dict(Qo=at(0) + 256, qos=768), BAD), (dict(Qo=at(0), qos=640), BAD), (dict(Qo=at(0) + 2 * 640, qos=768, Hq=1), BAD),
    (dict(Qo=at(1) - 16), BAD), (dict(Qo=at(2)), BAD), (dict(Qo=at(3)), BAD), (dict(Qo=at(5)), BAD), (dict(Qo=at(6)), BAD),
    (dict(vp=at(5)), BAD), (dict(kp=at(0)), BAD), (dict(vsc=at(1)), BAD), (dict(ksc=at(3) + 8), BAD), (dict(vp=at(2)), BAD),
], ids=str)
def test_append_refusals(lib, kw, want):
    assert _append(lib, **kw) == want


def test_binding_rejects_host_tensors(lib):
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    f, _ = pkg.attn_rope_freqs(64, device="cpu")
    with pytest.raises(TypeError, match="Q must be a CUDA tensor"):
        pkg.attn_rope(x, x, f)
    with pytest.raises(TypeError, match="dQ must be a CUDA tensor"):
        pkg.attn_rope_bwd(x, None, f)
    i, s = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    pages, one = torch.zeros(4, 3, 16, 64, dtype=torch.uint8), torch.ones(4, 3)
    with pytest.raises(TypeError, match="K must be a CUDA tensor"):
        pkg.attn_kv_append_rope_fp8(x, x, x, i, s, f, pages, one, pages, one)
    assert math.isfinite(float(f[0]))
