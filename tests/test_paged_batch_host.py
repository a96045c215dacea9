"""The paged operators' reading of a ragged batch (csrc/fa_paged.cuh) on the host, no GPU: the header's
functions compiled into a small program."""
import os
import subprocess

import pytest

from quantized_kv_cache_sm_gb300 import build as fa_build

CAP = 96

POSITIONS = r"""
#include <cstdio>
#include <cstdlib>
#include "fa_paged.cuh"
int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3)
    std::printf("%d\n", fa::row_position(std::atoi(argv[i]), std::atoll(argv[i + 1]),
                                         std::atoi(argv[i + 2])));
}
"""


@pytest.fixture(scope="module")
def row_position(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_batch")
    src, exe = d / "positions.cu", d / "positions"
    src.write_text(POSITIONS)
    subprocess.run([fa_build.nvcc_path(), "-std=c++17", *fa_build.ARCH, "-I", fa_build.CSRC, "-o", str(exe),
                    str(src)], check=True, capture_output=True)

    def call(cases):
        out = subprocess.run([str(exe), *(str(x) for c in cases for x in c)], check=True,
                             capture_output=True, text=True).stdout
        return [int(x) for x in out.split()]

    return call


def test_row_positions(row_position):
    """Rows of lengths that the table holds are at length - rows before the end; every other length,
    to the ends of 32 bits, gives a negative position (near -2^31 a difference of 32 bits would wrap to
    a large one)."""
    lens = [0, 1, 5, CAP - 1, CAP, CAP + 1, -1, -5, 2 ** 30, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1,
            -2 ** 31 + 6, -2 ** 31 + 7, -2 ** 30]
    cases = [(n, CAP, back) for n in lens for back in (1, 2, 7, 2 ** 30)]
    for (n, cap, back), got in zip(cases, row_position(cases), strict=True):
        if 0 <= n <= cap and n >= back:
            assert got == n - back
        else:
            assert got < 0, (n, back)
