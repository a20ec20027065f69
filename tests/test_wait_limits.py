"""The forms of the dense kernels' bounded wait end at their limit, each by itself, for all lanes of a warp where the
warp waits, and are reported (a short wait on a barrier that nothing completes; the context stays usable)."""

import pytest
import torch

import exact_attention_95_gb300 as pkg


@pytest.mark.gpu
@pytest.mark.parametrize("ms", [20, 150])
def test_every_form_of_wait_ends_at_its_limit(ms):
    pkg.attn_last_device_status()
    assert pkg.attn_selftest_wait_timeout(10 ** 5) == pkg.ATTN_OK  # (the kernel's first launch loads it)
    assert pkg.attn_last_device_status() == pkg.ATTN_ERR_TIMEOUT
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    assert pkg.attn_selftest_wait_timeout(ms * 10 ** 6) == pkg.ATTN_OK
    b.record()
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_ERR_TIMEOUT
    assert pkg.attn_last_device_status() == pkg.ATTN_OK
    assert 0.9 * ms <= a.elapsed_time(b) <= 2 * ms + 20  # (a try may take a while; launches beside it)
