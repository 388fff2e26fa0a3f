"""What a row of qsa_biased_gqa sees, from the kernels' own function compiled for
the host, against whole numbers without bounds (CPU only)."""

import itertools
import os
import subprocess

import pytest

from learned_sparse_attention_gb300 import build as B

LOW, HIGH = -2 ** 31, 2 ** 31 - 1
MOST = HIGH - 255  # tokens of a table row, at the most

SOURCE = r"""
#include <cstdio>
#include "row_output.cuh"
int main() {
  int p, window, doc, prefix;
  while (std::scanf("%d %d %d %d", &p, &window, &doc, &prefix) == 4) {
    const qsa::Span s = qsa::span_at(p, window, doc, prefix);
    std::printf("%d %d %d\n", s.p, s.lo, s.hi);
  }
}
"""

POSITIONS = [-1, 0, 1, 700, MOST - 1, MOST]  # as the kernels clamp them
WINDOWS = [0, 1, 100, HIGH - 1, HIGH]
ENDS = [LOW, LOW + 1, LOW + 256, -1, 0, 1, 500, 701, 5000, MOST - 1, MOST, MOST + 1, HIGH - 1, HIGH]


@pytest.fixture(scope="module")
def spans(tmp_path_factory):
    d = tmp_path_factory.mktemp("spans")
    (d / "spans.cu").write_text(SOURCE)
    exe = str(d / "spans")
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", B.INCLUDE, "-I", B.CSRC, str(d / "spans.cu"),
                    "-o", exe], check=True, capture_output=True)

    def ask(cases):
        text = "".join("%d %d %d %d\n" % c for c in cases)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def test_ends_of_the_integers(spans):
    cases = list(itertools.product(POSITIONS, WINDOWS, ENDS, ENDS))
    got = spans(cases)
    assert len(got) == len(cases)
    for (p, window, doc, prefix), (gp, lo, hi) in zip(cases, got):
        what = (p, window, doc, prefix, gp, lo, hi)
        if p < 0:
            assert gp == -1 and lo > hi and hi == -1, what
            continue
        # (no table has a token from MOST on)
        first, last = max(doc, 0, p - window + 1), max(p, min(prefix, MOST) - 1)
        assert gp == p, what
        assert (lo <= hi) == (first <= last), what
        # what follows counts tokens up to hi + 1 and tiles up to hi + 128
        assert 0 <= lo and 0 <= hi <= MOST, what
        if lo <= hi:
            assert lo == first and hi == last, what
