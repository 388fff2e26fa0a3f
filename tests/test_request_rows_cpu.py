"""Which rows a query_start_loc names, from the kernels' own function compiled for
the host (CPU only)."""

import itertools
import subprocess

import pytest

from learned_sparse_attention_gb300 import build as B

SOURCE = r"""
#include <cstdio>
#include "stage_helpers.cuh"
int main() {
  int start, end, rows;
  while (std::scanf("%d %d %d", &start, &end, &rows) == 3) std::printf("%d\n", qsa::rows_of_request(start, end, rows));
}
"""

LOW, HIGH = -2 ** 31, 2 ** 31 - 1
STARTS = [LOW, LOW + 1, LOW + 9, -10, -1, 0, 1, 63, 64, 65, 1000, 1 << 30, HIGH - 9, HIGH - 1, HIGH]


@pytest.fixture(scope="module")
def count(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "rows.cu").write_text(SOURCE)
    exe = str(d / "rows")
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", B.INCLUDE, "-I", B.CSRC, str(d / "rows.cu"),
                    "-o", exe], check=True, capture_output=True)

    def ask(cases):
        text = "".join("%d %d %d\n" % c for c in cases)
        return list(map(int, subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout.split()))
    return ask


def test_starts_of_every_kind(count):
    """A start far behind a later one (2^31 - 1, then -10) is no long request."""
    cases = list(itertools.product(STARTS, STARTS, [0, 1, 64, 65, HIGH]))
    for (start, end, rows), n in zip(cases, count(cases)):
        assert n == (end - start if 0 <= start <= end <= rows else -1), (start, end, rows, n)
