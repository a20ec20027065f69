"""Plain 64-bit implementation of the paged 8-bit cache, for its tests: the
tables of a step, the quantizing append and attention over the pages, written
from their definitions (loops over requests, numpy float64)."""

import numpy as np

from oracle import fp8


def tables(cached, added, free, table, page, T):
    """(table, kv_lens, cu, slots, positions, taken) as attn_kv_tables defines them."""
    table = table.copy()
    R, width = table.shape
    lens, cu = np.zeros(R, np.int64), np.zeros(R + 1, np.int64)
    slots, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    upto = at = taken = refused = 0
    for r in range(R):
        c, a = max(int(cached[r]), 0), max(int(added[r]), 0)
        have, full = -(-c // page), -(-(c + a) // page)
        first, at = at, at + a
        fits = full <= width and at <= T
        need = full - have if full <= width else 0
        upto += need
        served = fits and (need == 0 or upto <= len(free))
        cu[r + 1] = min(at, T)
        lens[r] = c + a if served else c
        if not served:
            refused += 1
            continue
        if need:
            table[r, have:full] = free[upto - need:upto]
            taken = max(taken, upto)
        for i in range(a):
            p = c + i
            slots[first + i] = int(table[r, p // page]) * page + p % page
            pos[first + i] = p
    return table, lens, cu, slots, pos, np.array([taken, refused])


def power_scale(amax):
    """The smallest 2^k, k >= -126, with amax <= 448 * 2^k."""
    k = -126
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def append(X, slots, codes, scales):
    """Appends X [T, Hkv, d] (float64 of the stored bf16) to copies of codes and scales."""
    codes, scales = codes.copy(), scales.astype(np.float64).copy()
    num_pages, Hkv, page, _ = codes.shape
    runs, before = [], None
    for t, s in enumerate(int(v) for v in slots):
        if 0 <= s < num_pages * page:
            if runs and before is not None and s == before + 1 and s % page:
                runs[-1][1] += 1
            else:
                runs.append([t, 1])
            before = s
        else:
            before = None
    for t, n in runs:
        p, off = divmod(int(slots[t]), page)
        for h in range(Hkv):
            x = X[t:t + n, h]
            fin = np.abs(x[np.isfinite(x)])
            s = power_scale(fin.max() if fin.size else 0.0)
            old = scales[p, h]
            if off > 0:
                s = max(s, old)
                if s > old:
                    v = fp8.decode_e4m3(codes[p, h, :off])
                    again = fp8.encode_e4m3(fp8.round_e4m3(np.where(np.isnan(v), 0.0, v) * (old / s)))
                    codes[p, h, :off] = np.where(np.isnan(v), codes[p, h, :off], again)
            nan = np.isnan(x)
            y = np.where(nan, 0.0, np.clip(x, -1e300, 1e300)) / s
            c = fp8.encode_e4m3(fp8.round_e4m3(y))
            codes[p, h, off:off + n] = np.where(nan, 0x7F, c)
            scales[p, h] = s
    return codes, scales


def dequantize(codes, scales, row, length):
    """[Hkv, length, d]: the first `length` tokens of the pages in `row`."""
    page = codes.shape[2]
    ids = np.asarray(row[:-(-length // page)], dtype=np.int64)
    v = fp8.decode_e4m3(codes[ids]) * scales[ids].astype(np.float64)[:, :, None, None]
    return v.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :length]


def attention(Q, kc, ks, vc, vs, table, cu, lens, scale, causal):
    """O, LSE, and the sums that bound the kernel's error: A = sum_j p_j |v_j| (per
    column); B = max_j scale * sum_c |q_c k_jc| and B[1] the same with max |q| for
    every q_c (per row).  Rows of no request: NaN."""
    T, Hq, d = Q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    O, A = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    LSE, B = np.full((T, Hq), np.nan), np.full((2, T, Hq), np.nan)
    for r in range(len(lens)):
        a, b, L = int(cu[r]), int(cu[r + 1]), int(lens[r])
        if b == a:
            continue
        k, v = dequantize(kc, ks, table[r], L), dequantize(vc, vs, table[r], L)
        for i in range(a, b):
            n = max(0, min(L, L - (b - a) + (i - a) + 1)) if causal else L
            for h in range(Hkv):
                q = Q[i, h * G:(h + 1) * G]
                out = slice(h * G, (h + 1) * G)
                if n == 0:
                    O[i, out], A[i, out], B[:, i, out], LSE[i, out] = 0.0, 0.0, 0.0, -np.inf
                    continue
                x = scale * (q @ k[h, :n].T)
                m = x.max(1, keepdims=True)
                e = np.exp(x - m)
                z = e.sum(1, keepdims=True)
                O[i, out] = e @ v[h, :n] / z
                A[i, out] = e @ np.abs(v[h, :n]) / z
                LSE[i, out] = (m + np.log(z))[:, 0]
                B[0, i, out] = scale * (np.abs(q) @ np.abs(k[h, :n]).T).max(1)
                B[1, i, out] = scale * np.abs(q).max(1) * np.abs(k[h, :n]).sum(1).max()
    return O, LSE, A, B


def bounds(O, LSE, A, B, d, bf16_out):
    """How far the kernels' O and LSE may be off.

    The products q k are exact in f16 operands; their fp32 sum over d terms is
    off by at most d * 2^-23 of the sum of magnitudes, the scaled logit in log2
    units by a few more half steps (2^-24 each) of its own size, together
    (d + 8) * 2^-23 * B[0].  Where q is the sum of two e4m3 numbers, an element
    is off by at most half of e4m3's smallest step, 2^-10, with the row's largest
    scaled above 224: 2^-10 / 224 * B[1].  e is the sum of the two.  A weight is then off by 2 e relative (its own
    logit and the maximum's), by the exponential's 2^-21, and by f16's half
    step 2^-11; the weights' sum by the first two.  fp32 sums of positive
    terms over lanes and warps add less than 2^-16.  bf16 output: 2^-8."""
    e = (d + 8) * 2.0 ** -23 * B[0] + 2.0 ** -10 / 224 * B[1]
    w = (2.0 ** -11 + 4 * e + 2.0 ** -20 + 2.0 ** -16)[..., None]
    tol_o = w * A + (2.0 ** -8 * (np.abs(O) + w * A) if bf16_out else 2.0 ** -23 * np.abs(O)) + 1e-30
    fin = np.where(np.isfinite(LSE), np.abs(LSE), 0.0)
    tol_l = 2 * e + 2.0 ** -16 + 2.0 ** -22 * fin
    return tol_o, tol_l


def bf16_bits(x):
    """Nearest bf16 (ties to even) of finite float32 values, as uint16."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
