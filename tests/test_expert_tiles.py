"""The split of an expert's rows into tiles, as the kernels compute it, over the whole range of row counts."""
import ctypes
import os
import subprocess

import pytest

from combine_warp_top_router_b200 import build

MOST_ROWS = 2 ** 31 - 4096  # rows of a call stay below


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("tiles")
    src, so = os.path.join(d, "tiles.cpp"), os.path.join(d, "tiles.so")
    with open(src, "w") as f:
        f.write('#include "ragged.cuh"\n'
                'extern "C" int tiles(int c, int most) { return md::ragged_tiles(c, most); }\n'
                'extern "C" int each(int c, int most, int gran) { return md::ragged_rows(c, most, gran); }\n')
    subprocess.run(["g++", "-O1", "-fwrapv", "-shared", "-fPIC", f"-I{build.CSRC}", src, "-o", so], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("most,gran", [(64, 16), (256, 32)])  # the few-row form's and the pairs'
def test_rows_are_covered_by_equal_tiles(split, most, gran):
    counts = list(range(0, 3000)) + [2 ** p + d for p in range(12, 31) for d in (-257, -256, -1, 0, 1, 255, 257)]
    counts += [MOST_ROWS - 1 - d for d in (0, 1, 31, 255, 4096, 2 ** 23, 2 ** 23 + 1, 2 ** 25, 2 ** 25 + 1)]
    for c in counts:
        n, each = split.tiles(c, most), split.each(c, most, gran)
        assert n == -(-c // most)
        if c == 0:
            assert each == 0
            continue
        assert each == -(-(-(-c // n)) // gran) * gran, c
        assert each <= most and (n - 1) * each < c <= n * each, c  # every tile has a row, and all rows a tile
