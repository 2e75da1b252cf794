"""The rows of a packed sequence (row_span of common.cuh, which every packed kernel asks), compiled for the host and
compared with the same rule in unbounded integers, at offsets, totals and bounds up to 2^31 - 1."""
import os
import subprocess

import pytest

from gated_deltanet_linear_18_b200 import _build

MAIN = r"""
#include <stdio.h>
#include "common.cuh"
int main() {
  int cu[2], T, most;
  while (scanf("%d %d %d %d", &cu[0], &cu[1], &T, &most) == 4) {
    const gdn::RowSpan sp = gdn::row_span(cu, 0, T, most);
    printf("%ld %d\n", sp.row0, sp.len);
  }
}
"""
MOST = 2 ** 31 - 1


def span(first, last, T, most):
    a = min(max(first, 0), T)
    return a, max(min(max(last, a), T, a + most) - a, 0)


@pytest.fixture(scope="module")
def row_span(tmp_path_factory):
    d = tmp_path_factory.mktemp("row_span")
    src, exe = d / "row_span.cu", d / "row_span"
    src.write_text(MAIN)
    subprocess.check_call([_build.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17",
                           "--expt-relaxed-constexpr", "-I", _build.CSRC, "-o", os.fspath(exe), os.fspath(src)])

    def run(cases):
        out = subprocess.run([os.fspath(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), text=True,
                             stdout=subprocess.PIPE, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def test_rows_of_a_packed_sequence(row_span):
    edges = [0, 1, 5, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 1, MOST - 1, MOST]
    cases = [(a, b, T, most) for T in edges for most in edges for a in [-3] + edges for b in [-3] + edges]
    for case, got in zip(cases, row_span(cases), strict=True):
        assert got == span(*case), case
