"""What the smoke check takes for the masks of a forward and its backward, on masks that are made here: right ones, and
those of a backward (or a forward) with a mistake."""

import os
import sys

import numpy as np
import pytest

import dropout as plain

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import __graft_entry__ as entry  # noqa: E402

SEED, OFFSET, P, B, H, N, D = 0x5320, 1, 0.25, 1, 4, 200, 128


def _weights(seed=SEED, offset=OFFSET, p=P, first=0):
    """[B, H, D, D]: the rows and keys from `first` on, as weights of 1 / N times their factors."""
    r = plain.factors(seed, offset, p, B, H, N).numpy() / N
    return r[:, :, first:first + D, first:first + D]


def _check(O, back):
    return entry.check_masks(O, np.ascontiguousarray(back.swapaxes(2, 3)), P, N)


@pytest.mark.parametrize("first", [0, N - D])
def test_the_same_mask_passes(first):
    w = _weights(first=first)
    assert abs(_check(w * (1 + 2.0 ** -8), w * (1 - 2.0 ** -8)) - 0.75) < 0.01


@pytest.mark.parametrize("wrong", [
    lambda w: _weights(offset=OFFSET + 1), lambda w: _weights(seed=SEED + 1), lambda w: _weights(seed=0, offset=0),
    lambda w: _weights(first=1), lambda w: np.roll(w, 1, 1), lambda w: w.swapaxes(2, 3),
    lambda w: np.full_like(w, 1 / N), lambda w: np.full_like(w, w.max()), lambda w: w * 0.75, lambda w: np.zeros_like(w),
], ids=["offset", "seed", "no rng", "rows and keys moved", "heads", "transposed", "no dropout", "nothing dropped", "no factor",
        "nothing kept"])
def test_a_backward_with_a_mistake_fails(wrong):
    w = _weights()
    with pytest.raises(RuntimeError, match="dropout"):
        _check(w, wrong(w))


@pytest.mark.parametrize("wrong", [lambda: _weights(p=0.5), lambda: np.repeat(_weights()[:, :1], H, 1),
                                   lambda: np.full((B, H, D, D), 1 / N)], ids=["probability", "one head's mask", "no dropout"])
def test_a_mistake_of_both_fails(wrong):
    w = wrong()
    with pytest.raises(RuntimeError, match="dropout"):
        _check(w, w)
