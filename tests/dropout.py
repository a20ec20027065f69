"""Plain 64-bit implementation of attention with dropout, for its tests (torch on any
device), and how far the kernels may be off."""

import math

import torch

M32 = 0xFFFFFFFF


def product(a, b):
    """(high, low) words of products of 32-bit numbers held in int64."""
    p = a * b  # wraps at 2^64, which both words survive
    return (p >> 32) & M32, p & M32


def philox(c, k, rounds=7):
    """Philox4x32 of counters c (four tensors) under the key k (two)."""
    c, k = list(c), list(k)
    for _ in range(rounds):
        h0, l0 = product(c[0], 0xD2511F53)
        h1, l1 = product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def numbers(seed, offset, B, Hq, N, device="cpu"):
    """u of attn_fwd_dropout's description: int64 [B, Hq, N, N]."""
    groups = -(-N // 32)
    shape = (B * Hq, N, groups)
    row = torch.arange(N, device=device)[None, :, None].expand(shape)
    head = torch.arange(B * Hq, device=device)[:, None, None].expand(shape)
    g = torch.arange(groups, device=device).expand(shape)
    off = torch.full(shape, offset & M32, device=device)
    key = [torch.tensor(v, device=device) for v in (seed & M32, (seed >> 32) & M32)]
    words = [w for half in (0, 1) for w in philox((row, 2 * g + half, head, off), key)]
    bit = torch.arange(32, device=device)
    u = sum(((w[..., None] >> bit) & 1) << k for k, w in enumerate(words))
    return u.reshape(B, Hq, N, 32 * groups)[..., :N]


def threshold(p):
    return math.floor(256 * p + 0.5)


def factors(seed, offset, p, B, Hq, N, device="cpu"):
    """What each element of the softmax is multiplied with."""
    T = threshold(p)
    return (numbers(seed, offset, B, Hq, N, device) >= T).double() / (1 - T / 256)


def forward(Q, K, V, r, scale, causal):
    """O, LSE, P in 64 bits, and what bounds the kernels' error: A = sum_j P r |v_j| (per column), e: by
    how much a weight's logarithm may be off (per row)."""
    G, N, d = Q.shape[1] // K.shape[1], Q.shape[2], Q.shape[3]
    q, k, v = Q.double(), K.double().repeat_interleave(G, 1), V.double().repeat_interleave(G, 1)
    x = torch.matmul(q, k.transpose(2, 3)) * scale
    size = torch.matmul(q.abs(), k.abs().transpose(2, 3)) * scale
    if causal:
        late = torch.ones(N, N, dtype=torch.bool, device=Q.device).triu(1)
        x, size = x.masked_fill(late, -math.inf), size.masked_fill(late, 0.0)
    lse = torch.logsumexp(x, -1)
    P = torch.exp(x - lse[..., None])
    # fp32 sums of d products, a logit's and its maximum's; log2 units' roundings are relative to the logits.
    e = (2 * (d + 8) * 2.0 ** -23 * size.amax(-1) + 2.0 ** -22 * lse.abs() + 2.0 ** -16)[..., None]
    return torch.matmul(P * r, v), lse, P, torch.matmul(P * r, v.abs()), e


HALF = 2.0 ** -8  # bf16's half step, relative


def forward_bounds(O, lse, A, e, bf16_out):
    """A weight is off by its logit and by bf16's half step; the divisor's sum takes the largest weight's
    rounding with it, which that weight may have kept for itself where it is dropped: another half step."""
    tol = (2 * HALF + 2 * e + 2.0 ** -16) * A
    return tol + ((HALF * (O.abs() + tol)) if bf16_out else 2.0 ** -23 * O.abs()) + 1e-30, (e + 2.0 ** -20)[..., 0]


def backward(Q, K, V, O, dO, r, scale, causal):
    """[(gradient, bound)] of Q, K, V in 64 bits, O being an input; the bounds are per element."""
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    _, _, P, _, e = forward(Q, K, V, r, scale, causal)
    q, k, v = Q.double(), K.double().repeat_interleave(G, 1), V.double().repeat_interleave(G, 1)
    g, o = dO.double(), O.double()
    t = torch.matmul
    D, Dsize = (g * o).sum(-1, keepdim=True), (g * o).abs().sum(-1, keepdim=True)
    dP, dPsize = t(g, v.transpose(2, 3)) * r, t(g.abs(), v.abs().transpose(2, 3)) * r
    dS = P * (dP - D)
    # dS: its own rounding to bf16, P's relative error, and fp32 sums of d terms in dP and D.
    sums = (d + 8) * 2.0 ** -23
    s_off = (HALF + 2 * e) * dS.abs() + P * (1 + HALF) * sums * (dPsize + Dsize)
    p_off = (HALF + 2 * e) * P * r

    def of_group(x):
        return x.reshape(B, Hkv, G, *x.shape[2:]).sum(2)

    out = [(scale * t(dS, k), scale * t(s_off, k.abs()), scale * t(dS.abs(), k.abs())),
           (scale * of_group(t(dS.transpose(2, 3), q)), scale * of_group(t(s_off.transpose(2, 3), q.abs())),
            scale * of_group(t(dS.abs().transpose(2, 3), q.abs()))),
           (of_group(t((P * r).transpose(2, 3), g)), of_group(t(p_off.transpose(2, 3), g.abs())),
            of_group(t((P * r).transpose(2, 3), g.abs())))]
    # fp32 sums over rows or keys (2^-23 of the sizes for each of up to N * G / 16 products), and the result's rounding.
    many = (N * G / 16 + 16) * 2.0 ** -23
    return [(x, off + many * size + HALF * (x.abs() + off) + 1e-30) for x, off, size in out]
