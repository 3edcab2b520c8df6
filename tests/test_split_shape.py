"""Shared memory of the split-K INT8 GEMM, on the CPU: the header's own arithmetic, compiled with
the host compiler and printed for every number of tokens, width and split.

A CTA that is resident must find its tensor memory free: an SM has 512 columns, and an allocation
that does not fit waits without a limit for another CTA's, whose cluster may be waiting for this
one. So whatever mix of these CTAs an SM's shared memory holds, from one call or several at once,
has to hold at most 512 columns."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "w4a8_ptq_linear_b200", "csrc")
SM, BLOCK, LIMIT, COLUMNS = 228 * 1024, 1024, 227 * 1024, 512

PROGRAM = r"""
#include <cstdio>
#include "split_shape.h"
int main() {
  for (int T = 1; T <= 256; ++T)
    for (int K = 32; K <= 32768; K = K < 2048 ? K + 32 : K + 1056)
      for (int S = 1; S <= oq::kSplitMax; ++S) {
        const oq::SplitShape c = oq::split_shape(T, K, S);
        if (c.ks)
          std::printf("%d %d %d %d %d %d %d %d %d\n", T, K, S, c.npad, c.tcols, c.ks, c.ns, c.off_bar,
                      c.smem);
      }
}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    src, exe = str(d / "s.cpp"), str(d / "s")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, src, "-o", exe], check=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()
    return sorted({tuple(map(int, l.split()))[3:] + (int(l.split()[1]), int(l.split()[2]))
                   for l in lines})


def test_no_mix_of_ctas_asks_for_more_tensor_memory_than_an_sm_has(shapes):
    least = {}   # columns -> the least shared memory that comes with them
    for _, tcols, _, _, _, smem, _, _ in shapes:
        least[tcols] = min(least.get(tcols, SM), smem + BLOCK)
    assert set(least) == {32, 64, 128, 256}
    # the most columns that fit an SM's shared memory, by every mix
    kinds = sorted(least.items())

    def most(i, room):
        if i == len(kinds):
            return 0
        cols, smem = kinds[i]
        return max(n * cols + most(i + 1, room - n * smem) for n in range(room // smem + 1))

    assert most(0, SM) <= COLUMNS


def test_ring_and_partial_sums_fit(shapes):
    for npad, tcols, ks, ns, off_bar, smem, K, S in shapes:
        assert npad % 16 == 0 and tcols >= npad and tcols & (tcols - 1) == 0
        assert 1 <= ns <= min(ks, 12) and off_bar % 1024 == 0
        assert off_bar >= ns * (128 + npad) * 128 and off_bar >= npad * 128 * 4
        assert off_bar + 256 + 12 * 256 + 1024 <= smem <= LIMIT
        nkb = (K + 127) // 128
        assert (S - 1) * ks < nkb <= S * ks   # every CTA has a block of K, all are taken
