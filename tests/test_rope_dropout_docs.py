"""What the header and the docstrings say of frequencies from elsewhere, of probabilities at the ends, and of a workspace
for several calls."""

import math

import pytest
import torch

import exact_attention_95_gb300 as pkg
from exact_attention_95_gb300 import build as libbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return pkg.load_library()


@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 500000.0), (2, 10000.0)])
def test_frequencies_from_radians(rot, base):
    w = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    made = (w / (2 * math.pi) * 2.0 ** 64).round().long()
    freqs, _ = pkg.attn_rope_freqs(rot, base, device="cpu")
    # A few operations in 64 bits on either side (2^-53 each, a power's exponent magnified by its logarithm, below 32).
    assert ((made - freqs).double().abs() <= 64 * 2.0 ** -53 * freqs.double() + 1).all()
    # Slower ones than half a turn a position fit: the fastest that does not is pi.
    assert int((torch.tensor([3.14159], dtype=torch.float64) / (2 * math.pi) * 2.0 ** 64).round().long()) > 0


def test_the_workspace_does_not_grow_with_the_length():
    sizes = {N: pkg.attn_bwd_dropout_workspace_size(1, 32, 8, N, 128, True) for N in (2000, 2432, 2560)}
    assert sizes[2000] > sizes[2432] and sizes[2560] >= sizes[2432]


@pytest.mark.gpu
def test_the_largest_of_several_sizes_serves_them_all():
    lengths, B, Hq, Hkv, d = (40, 700, 2000, 2432), 1, 32, 8, 128
    ws = torch.empty(max(pkg.attn_bwd_dropout_workspace_size(B, Hq, Hkv, N, d, True) for N in lengths), dtype=torch.uint8,
                     device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rng = torch.tensor([5, 6], device="cuda")
    for N in lengths:
        Q, K, V, dO = (torch.randn(B, h, N, d, generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv, Hq))
        O, L = pkg.attn_fwd_dropout(Q, K, V, 0.1, rng, None, True)
        _, dK, dV = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, 0.1, rng, None, True, workspace=ws)
        _, dK2, dV2 = pkg.attn_bwd_dropout(Q, K, V, O, dO, L, 0.1, rng, None, True)
        assert torch.equal(dK, dK2) and torch.equal(dV, dV2)
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("p,drops", [(0.0, False), (1 / 512 - 1e-6, False), (1 / 512, True), (511 / 512 - 1e-6, True), (511 / 512, None)])
def test_probabilities_at_the_ends(p, drops):
    Q, K, V = (torch.randn(1, 2, 300, 64, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16() for _ in range(3))
    rng = torch.tensor([5, 6], device="cuda")
    if drops is None:
        with pytest.raises(pkg.AttnError):
            pkg.attn_fwd_dropout(Q, K, V, p, rng)
        return
    assert torch.equal(pkg.attn_fwd_dropout(Q, K, V, p, rng)[0], pkg.attn_fwd(Q, K, V)[0]) == (not drops)
