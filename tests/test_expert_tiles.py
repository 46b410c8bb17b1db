"""The split of an expert's rows into tiles, as the kernels compute it, over the whole range of row counts, and
the rule that chooses a call's kernel form."""
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
                'extern "C" int each(int c, int most, int gran) { return md::ragged_rows(c, most, gran); }\n'
                'extern "C" bool few(int64_t rows, int E, int64_t columns, int sub, int sms)\n'
                '{ return md::ragged_few(rows, E, columns, sub, sms); }\n')
    subprocess.run(["g++", "-O1", "-fwrapv", "-shared", "-fPIC", f"-I{build.CSRC}", src, "-o", so], check=True)
    h = ctypes.CDLL(so)
    h.few.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    h.few.restype = ctypes.c_bool
    return h


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


@pytest.mark.parametrize("E,per,columns,few", [
    (64, 64, 2048, True), (64, 65, 2048, False), (256, 1, 1024, True),            # by the weights' reads
    (1, 100, 512, True), (8, 72, 256, True), (4, 128, 2048, True),                # too few wide tiles for the GPU
    (1, 4096, 1024, False), (8, 2048, 256, False), (8, 256, 1024, False),         # and too many narrow ones
    (2, 8192, 256, False), (1, 2 ** 31 - 4097, 8, False)])
def test_which_form(split, E, per, columns, few):
    assert split.few(E * per, E, columns, 256, 148) == few
    assert split.few(E * per, E, columns // 2, 128, 148) == few  # the gated product: half as wide
