"""Plain 64-bit implementation of rotary positions, for their tests, and how far the
kernels may be off."""

import math

import numpy as np

import paged
from oracle import fp8


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """(turns a position of each pair, amplitude), as attn_rope_freqs defines them."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) / (2 * math.pi) for i in range(rot // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        keep = np.clip((f * original_len - low) / (high - low), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1
    return f, 1.0


def angles(positions, freqs):
    """2 pi frac(pos * freq / 2^64) for int positions [n] and freqs [rot / 2], in whole numbers up to the fraction."""
    turns = [[(int(p) * int(f)) % 2 ** 64 / 2.0 ** 64 for f in freqs] for p in positions]
    return 2 * math.pi * np.array(turns).reshape(len(positions), len(freqs))


def rotate(x, positions, freqs, interleaved, amplitude, sign=1.0):
    """x [n, heads, d] float64 with a position a row -> (rotated, sum of |x| of each element's pair times the
    amplitude, 0 where nothing turns)."""
    rot = 2 * len(freqs)
    y, size = x.copy(), np.zeros_like(x)
    pos = np.asarray(positions, dtype=np.int64)
    a = angles(np.maximum(pos, 0), freqs)[:, None, :]
    c, s = amplitude * np.cos(a), sign * amplitude * np.sin(a)
    i = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    j = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    on = (pos >= 0)[:, None, None]
    y[..., i] = np.where(on, x[..., i] * c - x[..., j] * s, x[..., i])
    y[..., j] = np.where(on, x[..., j] * c + x[..., i] * s, x[..., j])
    size[..., i] = size[..., j] = np.where(on, amplitude * (np.abs(x[..., i]) + np.abs(x[..., j])), 0.0)
    return y, size


# cos and sin are off by at most 2^-22; the amplitude's rounding, its product with them, the product
# with x2 and the sum add a half step (2^-24 relative) each of terms no larger than the pair's |x1| + |x2|
# times the amplitude: 2^-22 + 4 * 2^-24 < 2^-21 of it.
TURN = 2.0 ** -21


def tolerance(y, size, bf16):
    """Of a rotated element: TURN, and the result's rounding (which fp32's is a part of above)."""
    off = TURN * size
    return off + ((2.0 ** -8 * (np.abs(y) + off) + 2.0 ** -134) if bf16 else 2.0 ** -149)


def check_append(x, size, slots, before, scales_before, codes, scales):
    """Whether codes and scales are those that x [T, Hkv, d] (float64, off by TURN * size) gives when appended to
    (before, scales_before): every number within what numbers that far off give.  Asserts."""
    num_pages, Hkv, page, _ = codes.shape
    off_x = TURN * size
    assert np.isfinite(x).all()
    want_codes, known = before.copy(), np.ones(before.shape, bool)
    want_scales = scales_before.astype(np.float64).copy()
    runs, last = [], None
    for t, s in enumerate(int(v) for v in slots):
        if 0 <= s < num_pages * page:
            if runs and last is not None and s == last + 1 and s % page:
                runs[-1][1] += 1
            else:
                runs.append([t, 1])
            last = s
        else:
            last = None
    for t, n in runs:
        p, off = divmod(int(slots[t]), page)
        for h in range(Hkv):
            y, e = x[t:t + n, h], off_x[t:t + n, h]
            s = float(scales[p, h])
            lo = paged.power_scale(max(0.0, (np.abs(y) - e).max()))
            hi = paged.power_scale((np.abs(y) + e).max())
            if off > 0:
                lo, hi = max(lo, want_scales[p, h]), max(hi, want_scales[p, h])
            assert lo <= s <= hi, (p, h, s, lo, hi)
            if off > 0 and s > want_scales[p, h]:
                again = fp8.round_e4m3(fp8.decode_e4m3(before[p, h, :off]) * (want_scales[p, h] / s))
                want_codes[p, h, :off] = fp8.encode_e4m3(again)
            got = fp8.decode_e4m3(codes[p, h, off:off + n])
            assert (fp8.round_e4m3((y - e) / s) <= got).all() and (got <= fp8.round_e4m3((y + e) / s)).all(), (p, h)
            known[p, h, off:off + n] = False
            want_scales[p, h] = s
    assert np.array_equal(np.where(known, want_codes, 0), np.where(known, codes, 0))
    assert np.array_equal(want_scales, scales.astype(np.float64))
