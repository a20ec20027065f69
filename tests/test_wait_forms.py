"""Bounded waits in the sources of the dense kernels.  A wait that runs out must not part a warp's lanes:
TMEM loads and stores, shuffles and votes are for all of them at once, and the rest would wait for
those that left, or do what is not defined.  So outside of code that a single lane runs, a wait has
one result for its warp.  (Read, not run: a kernel whose waits run out is no test for a shared GPU.)"""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_95_gb300", "csrc")
KERNELS = ["fwd_persist.cu", "fwd_sm103.cu", "fp8.cu", "bwd_sm103.cu"]


def _block(text, start):
    """Index behind the brace that closes the one at `start`."""
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced braces")


def _whole_warps(name):
    """The source without comments and without what a single lane runs."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    single = re.compile(r"if \([^;{}|]*(?:\blane|threadIdx\.x) == 0\b[^;{}|]*\) \{")
    while m := single.search(text):
        text = text[:m.start()] + text[_block(text, m.end() - 1):]
    return text


def test_single_lanes_are_taken_out(tmp_path, monkeypatch):
    (tmp_path / "x.cu").write_text("a; if (warp == 0 && lane == 0) { mbar_wait(b); { c; } } mbar_wait(d); // mbar_wait(e)\n")
    monkeypatch.setattr("test_wait_forms.CSRC", str(tmp_path))
    assert re.findall(r"mbar_wait\((\w)", _whole_warps("x.cu")) == ["d"]


@pytest.mark.parametrize("name", KERNELS)
def test_warps_wait_as_one(name):
    text = _whole_warps(name)
    assert "tmem_ld" in text and "mbar_wait_warp(" in text
    assert re.findall(r"[^\n]*\bmbar_wait(?:_drain)?\([^\n]*", text) == []
