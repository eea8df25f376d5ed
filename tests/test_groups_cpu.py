"""Arithmetic of csrc/groups.h that the kernels of the MXFP4 experts rely on, at the ends of its ranges: the functions that
run on the GPU, compiled for the host."""

import os
import subprocess

import pytest

from block_scaled_fp8_amax_amd import _build

MAIN = r"""
#include "groups.h"
#include <stdio.h>
#include <stdlib.h>
using namespace fp8blk;
int main(int argc, char** argv) {
  for (int i = 2; i + 1 < argc; i += 2) {
    const int a = atoi(argv[i]), b = atoi(argv[i + 1]);
    switch (argv[1][0]) {
      case 's': printf("%d\n", stages_in(a, b)); break;
      case 'a': printf("%d\n", add_tiles(a, b)); break;
      case 't': printf("%d\n", times_tiles(a, b)); break;
    }
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("groups")
    (d / "main.hip").write_text(MAIN)
    subprocess.run([_build._hipcc(), "--cuda-host-only", "-std=c++17", "-O1", "-Wno-unused-function", "-I", _build.INCLUDE,
                    "-I", _build.CSRC, str(d / "main.hip"), "-o", str(d / "main")], check=True, capture_output=True, text=True)

    def run(what, pairs):
        args = [str(v) for p in pairs for v in p]
        out = subprocess.run([str(d / "main"), what, *args], check=True, capture_output=True, text=True,
                             env={**os.environ, "HIP_VISIBLE_DEVICES": ""})
        return [int(v) for v in out.stdout.split()]
    return run


def test_stages_up_to_the_most_rows(program):
    """A group may have all of total_m <= 2^31 - 1 rows: the number of its stages rounds up without passing 2^31."""
    pairs = [(p, e) for e in (32, 64) for p in (0, 1, 63, 64, 65, 2**31 - 65, 2**31 - 64, 2**31 - 63, 2**31 - 2, 2**31 - 1)]
    assert program("stages", pairs) == [-(-p // e) for p, e in pairs]


def test_tiles_are_counted_without_passing_an_int(program):
    """Offsets [0, m, 0, m, ...] give every second group all rows: 512 groups of up to 2^26 row tiles, of up to 2^18 column
    tiles each.  The running sums, in any order of addition, stay sorted and end at the most that is counted."""
    most = 2**30
    pairs = [(0, 0), (0, 5), (most - 1, 0), (most - 2, 1), (most - 1, 1), (most, most), (most, 0), (2**26, 2**26), (most - 7, 9)]
    assert program("add", pairs) == [min(a + b, most) for a, b in pairs]
    pairs = [(0, 3), (2**15, 2**15 - 1), (2**15, 2**15), (2**26, 2**18), (most, 2**18), (most, 1), (3, 0), (77, 99)]
    assert program("times", pairs) == [min(a * b, most) for a, b in pairs]
    sums = [2**26 * (g % 2) for g in range(1024)]       # as the kernels add them: in steps of 1, 2, 4, ... groups
    d = 1
    while d < len(sums):
        before = [0] * d + sums[:-d]
        sums = program("add", list(zip(sums, before)))
        d *= 2
    assert sums == sorted(sums) and sums[-1] == most and sums[:8] == [2**26 * ((g + 1) // 2) for g in range(8)]
