"""The divisor of attention with dropout.  A row's weights are rounded to bf16 where they multiply V; what
that takes from each tile's largest one is taken from the divisor too, which is right for a weight
that is kept and wrong for one that is dropped.  So it has to be done where most weights are kept, and not
where most are dropped."""

import math

import pytest
import torch

import exact_attention_95_gb300 as pkg

import dropout as plain

SEED, OFFSET = 0x0123456789ABCDEF, 7


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("p", [0.1, 0.4, 0.5, 0.9, 0.98])
def test_rows_held_by_one_weight(p, d):
    """Logits 0 at key 0, 5 at key `big` of the second tile, -40 else: the second tile's largest weight is e^5 (the
    running maximum stays where it was), which bf16 rounds by 0.28 %, and all others are 1 or nothing."""
    N, Hq, big = 512, 8, 130
    size = math.exp(5.0)
    assert abs(size - float(torch.tensor(size).bfloat16())) > 0.0025 * size
    Q, K, V = (torch.zeros(1, Hq, N, d) for _ in range(3))
    Q[..., 0] = 1.0
    K[..., 0] = -40.0
    K[:, :, 0, 0], K[:, :, big, 0] = 0.0, 5.0
    V[:, :, 0, 0] = V[:, :, big, 1] = 1.0
    Q, K, V = (t.bfloat16().cuda() for t in (Q, K, V))
    rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda")
    O, _ = pkg.attn_fwd_dropout(Q, K, V, p, rng, 1.0, False, torch.float32)
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK
    r = plain.factors(SEED, OFFSET, p, 1, Hq, N, "cuda")
    want, _, _, A, e = plain.forward(Q, K, V, r, 1.0, False)
    # Logits and the fp32 division: no rounding of a weight.
    tight = (2 * e + 2.0 ** -16) * A
    kept = r[..., big] > 0
    if plain.threshold(p) >= 128:
        # The weight 1 of key 0 is exact, and so is its quotient where the other one does not enter.
        rows = ~kept & (r[..., 0] > 0)
        assert rows.any() and ((O[..., 0] - want[..., 0]).abs() <= tight[..., 0])[rows].all()
    else:
        # The rounding that numerator and divisor share cancels.
        rows = kept
        assert rows.any() and ((O[..., 1] - want[..., 1]).abs() <= tight[..., 1])[rows].all()
    off = (plain.HALF + 2 * e + 2.0 ** -16) * A
    assert ((O - want).abs() <= off + 1e-30).all()
