"""Arrays of a call of the paged cache that share memory: refused before anything is
launched (no GPU needed)."""

import pytest

from test_paged_abi import BAD, P, _fwd, _tables, at, lib  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(slots=at(7), pos=at(7)),          # two outputs in one place
    dict(lens=at(5)),                      # kv_lens and cu_tokens
    dict(cu=P(0x900000 - 12)),             # the last of cu_tokens is taken[0]
    dict(taken=P(0x700000 + 32)),          # taken in the last slot
    dict(pos=at(3)), dict(lens=P(0x400000 + 44)), dict(slots=P(0x400000 - 32)),  # in the block table
], ids=str)
def test_tables_refuse_outputs_over_one_another(lib, kw):  # noqa: F811
    assert _tables(lib, **kw) == BAD


@pytest.mark.parametrize("kw", [
    dict(O=at(0)),                                            # in place of Q
    dict(O=P(0x100000 + 4 * 4096 * 2 + 4096 * 2 - 16)),       # over Q's last elements
    dict(O=at(1)), dict(L=at(3)), dict(L=at(2)), dict(O=at(4)), dict(L=P(0x600000 + 44)), dict(L=P(0x700000 - 4)),
    dict(L=at(7)), dict(L=at(8)), dict(ws=at(9)), dict(ws=P(0x900000 - 256)), dict(ws=at(3)),
    dict(O=P(0xb00000 + 4096), out=1),
], ids=str)
def test_attention_refuses_outputs_over_another_array(lib, kw):  # noqa: F811
    assert _fwd(lib, **kw) == BAD
