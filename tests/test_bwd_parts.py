"""Where the dropout backward's parts of dK and dV lie: the index arithmetic of the kernels, compiled for the
host, against the workspace's size, and the debug variant's checks of those indices in the sources."""

import os
import re
import subprocess

import pytest

import exact_attention_95_gb300 as pkg
from exact_attention_95_gb300 import build as libbuild

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_95_gb300", "csrc")

# What a part's CTAs write, float4 by float4: 1 where one is written twice or outside, 2 where one that is read was not written.
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "kernels.h"
using namespace attn;
template <int D>
int run(BwdParams p) {
  std::vector<char> written(p.parts_f4, 0);
  const int tiles = p.Npad / kBwdKeys, G = p.Hq / p.Hkv;
  for (int split = 0; split < p.q_splits; ++split)
    for (int bhk = 0; bhk < p.B * p.Hkv; ++bhk)
      for (int key = 0; key < p.N; ++key)
        for (int which = 0; which < 2; ++which)
          for (int col = 0; col < D; col += 32)  // the epilogue's pieces, eight float4 each
            for (int i = 0; i < 8; ++i) {
              const size_t at = split * part_stride<D>(p) + part_at<D>(p, which, bhk, key, col / 4) + i * kBwdKeys;
              if (at >= p.parts_f4 || written[at]) return 1;
              written[at] = 1;
            }
  for (int jt = 0; jt < tiles; ++jt)
    for (int bhk = 0; bhk < p.B * p.Hkv; ++bhk)
      for (int key = jt * kBwdKeys; key < p.N && key < (jt + 1) * kBwdKeys; ++key)
        for (int which = 0; which < 2; ++which)
          for (int piece = 0; piece < D / 16; ++piece)  // the join's, four
            for (int k = 0; k < p.q_splits; ++k)
              for (int c = 0; c < 4; ++c) {
                const size_t at = part_at<D>(p, which, bhk, key, 4 * piece) + k * part_stride<D>(p) + c * kBwdKeys;
                if (at >= p.parts_f4 || !written[at]) return 2;
              }
  return 0;
}
int main(int n, char** v) {
  BwdParams p{};
  p.B = atoi(v[1]), p.Hq = atoi(v[2]), p.Hkv = atoi(v[3]), p.N = atoi(v[4]), p.q_splits = atoi(v[6]);
  p.Npad = (p.N + kBwdKeys - 1) / kBwdKeys * kBwdKeys;
  p.parts_f4 = strtoull(v[7], nullptr, 10) / 16;
  return atoi(v[5]) == 128 ? run<128>(p) : run<64>(p);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("parts")
    (d / "parts.cu").write_text(PROGRAM)
    exe = str(d / "parts")
    r = subprocess.run([libbuild._nvcc(), *libbuild.ARCH, "-std=c++17", "-O1", "-I", CSRC, str(d / "parts.cu"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("B,Hq,Hkv,N,d,causal", [
    (2, 12, 4, 777, 128, True), (2, 12, 4, 777, 64, False), (1, 16, 1, 2000, 128, True), (1, 4, 4, 129, 64, True),
    (1, 8, 2, 1, 128, False), (1, 64, 1, 128, 128, False), (3, 2, 1, 640, 64, False),
])
def test_parts_fill_their_room_and_no_more(program, B, Hq, Hkv, N, d, causal):
    libbuild.build()
    room = (pkg.attn_bwd_dropout_workspace_size(B, Hq, Hkv, N, d, causal) - pkg.attn_bwd_workspace_size(B, Hq, Hkv, N, d))
    one = 2 * B * Hkv * -(-N // 128) * 128 * d * 4
    assert room % one == 0
    splits = room // one
    if splits:
        assert 2 <= splits
        args = [str(v) for v in (B, Hq, Hkv, N, d, splits)]
        assert subprocess.run([program, *args, str(room)], timeout=120).returncode == 0
        # The program sees a room that is too small.
        last = one - 128 * d * 4 + ((N - 1) % 128) * 16 + (d // 4 - 1) * 2048  # the last float4 of a part that is written
        assert subprocess.run([program, *args, str((splits - 1) * one + last)], timeout=120).returncode == 1


def test_the_debug_variant_checks_the_parts_indices():
    with open(os.path.join(CSRC, "bwd_sm103.cu"), encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    uses = [m.start() for m in re.finditer(r"reinterpret_cast<(?:const )?float4\*>\(p\.parts\)", text)]
    assert len(uses) == 2  # written, read
    for u in uses:
        before = text[:u].rsplit("dcheck(", 1)[1]
        assert len(before) < 250 and re.match(r"at \+ [^;]*< p\.parts_f4", before)
    # What is read is then stored as dK and dV.
    assert re.search(r"dcheck\(at \+ \(n - 1\) \* stride \+ 3 \* kBK < p\.parts_f4 && bhk \* p\.N \+ key < ", text)
