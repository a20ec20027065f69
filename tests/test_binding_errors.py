"""Errors of calls through the extension module are the library's, as without it."""

import pytest
import torch

import exact_attention_95_gb300 as pkg


@pytest.mark.gpu
@pytest.mark.parametrize("module", [True, False])
@pytest.mark.parametrize("d", [32, 96, 256])
def test_head_dimensions_without_a_kernel_are_unsupported(d, module, monkeypatch):
    if not module:
        monkeypatch.setattr(pkg, "_fast", False)
    Q, L = torch.zeros(1, 2, 8, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 2, 8, device="cuda")
    rng = torch.zeros(2, dtype=torch.int64, device="cuda")
    for call in (lambda: pkg.attn_fwd_dropout(Q, Q, Q, 0.1, rng), lambda: pkg.attn_bwd_dropout(Q, Q, Q, Q, Q, L, 0.1, rng),
                 lambda: pkg.attn_bwd(Q, Q, Q, Q, Q, L)):
        with pytest.raises(pkg.AttnError) as e:
            call()
        assert e.value.code == pkg.ATTN_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert pkg.attn_last_device_status() == pkg.ATTN_OK
