"""The delta rule's equal shares of all heads' chunks, on the host: which
(head, chunk) every block takes, on parts with more and with fewer SMs than a
GB300 (152), where the plan chooses shares from 153 heads on."""

import os
import subprocess

import pytest

from mamba_selective_scan_gb300 import build

SRC = r"""
#include <stdio.h>
#include <stdlib.h>
#include "m3_delta_tc.cuh"
int main(int argc, char** argv) {
  const int sms = atoi(argv[1]), heads = atoi(argv[2]), nc = atoi(argv[3]);
  const unsigned blocks = m3::delta_share_blocks(heads, sms);
  for (unsigned b = 0; b < blocks; ++b) {
    const m3::TcWalk w(true, heads, nc, b, blocks, 0, nc);
    for (int i = 0; i < w.n; ++i) {
      const m3::TcStep t = w.at(i);
      printf("%u %d %d %d %d %d %d\n", b, t.bh, t.c, t.first, t.last, t.take, t.give);
    }
  }
  return blocks > (unsigned)sms;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("walk")
    (d / "walk.cu").write_text(SRC)
    exe = str(d / "walk")
    subprocess.run([build.nvcc_path(), *build.ARCH_FLAGS, "-std=c++17", "-I", build.CSRC, "-o", exe, str(d / "walk.cu")],
                   check=True, capture_output=True)

    def run(sms, heads, nc):
        r = subprocess.run([exe, str(sms), str(heads), str(nc)], check=True, capture_output=True, text=True)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


@pytest.mark.parametrize("sms", [132, 148, 152, 160, 192])
@pytest.mark.parametrize("heads", [153, 159, 160, 161, 191, 305, 1000])
@pytest.mark.parametrize("nc", [1, 2, 5, 33])
def test_every_chunk_once_and_states_handed_over(walk, sms, heads, nc):
    steps = walk(sms, heads, nc)
    assert sorted((s[1], s[2]) for s in steps) == [(h, c) for h in range(heads) for c in range(nc)]
    runs, run = [], []  # (block, head, first chunk, last chunk, take, give)
    for b, h, c, first, last, take, give in steps:
        if run and not first:
            assert (b, h, c) == (run[0], run[1], run[3] + 1)
            run[3] = c
        else:
            assert first
            run = [b, h, c, c, take, give]
        if last:
            runs.append(tuple(run))
    begun = {r[1]: r for r in runs if r[2] == 0}
    first_of = {}
    for r in runs:
        first_of.setdefault(r[0], r)
    for b, h, c0, c1, take, give in runs:
        assert take == (c0 > 0) and give == (c1 < nc - 1)
        if take:  # from the block before, which does that part first, and no more than this block does before it
            other = begun[h]
            assert other[0] == b - 1 and other[5] and other[3] + 1 == c0 and first_of[other[0]] == other
            mine = [s[:3] for s in steps if s[0] == b]
            assert other[3] + 1 <= mine.index((b, h, c0)) + 1
