"""The attention's launch rule on the host: how many key tiles a piece of rows meets, and how many
CTAs share them."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_gqa_decode_04_gb300", "csrc")
GB300 = (152, 76, 36, 15)                  # clusters of 1, 2, 4 and 8 CTAs that fit at once

SOURCE = """
#include "attend_plan.h"
extern "C" int64_t tiles(int64_t max_len, int window, int group) {
    return pgd::attend::piece_tiles(max_len, window, group);
}
extern "C" int cluster(const int* f, int64_t units, int64_t tiles, int few, double us) {
    const int fit[4] = {f[0], f[1], f[2], f[3]};
    return pgd::attend::choose_cluster(fit, units, tiles, few, us);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I" + CSRC,
                    str(d / "plan.cpp"), "-o", str(d / "plan.so")], check=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    i64 = ctypes.c_int64
    lib.tiles.restype, lib.tiles.argtypes = i64, [i64, ctypes.c_int, ctypes.c_int]
    lib.cluster.argtypes = [ctypes.POINTER(ctypes.c_int), i64, i64, ctypes.c_int, ctypes.c_double]
    return lib


def cluster(plan, rows, group, hkv, max_len, window=0, us=1.2, fit=GB300):
    """Of a batch with these query tokens a sequence, as paged_gqa_attend asks for it."""
    total, B = sum(rows), len(rows)
    pieces = (total * group >> 8) + B
    few = total * group <= pieces * 128
    return plan.cluster((ctypes.c_int * 4)(*fit), pieces * hkv, plan.tiles(max_len, window, group),
                        few, us)


@pytest.mark.parametrize("group", [1, 3, 4, 8, 100, 256, 300])
@pytest.mark.parametrize("window", [1, 2, 37, 128, 129, 500])
def test_tiles_of_a_windowed_piece(plan, window, group):
    """No piece meets more tiles than the bound, and some piece meets that many or one fewer."""
    most = 0
    for offset in range(130):              # position of the sequence's first query
        for row0 in (0, 256, 512, 768):
            p0, p1 = offset + row0 // group, offset + (row0 + 255) // group
            p0, p1 = p0 + 1024, p1 + 1024  # behind tokens enough for every window
            most = max(most, p1 // 128 - (p0 - window + 1) // 128 + 1)
    bound = plan.tiles(1 << 20, window, group)
    assert most <= bound <= most + 1


def test_tiles_without_a_window_or_with_a_wide_one(plan):
    for n in (1, 127, 128, 129, 5000):
        assert plan.tiles(n, 0, 4) == -(-n // 128)
        assert plan.tiles(n, 1 << 30, 4) == -(-n // 128)


def test_a_window_bounds_the_tiles_that_are_shared(plan):
    """A few queries with a window of 512 behind a table for 32768 or more: what a table of just
    the window would get, not eight CTAs for some five tiles."""
    for max_len in (32768, 131072, 1 << 24):
        for B in (2, 9, 40):
            want = cluster(plan, [4] * B, 4, 8, 700)
            assert cluster(plan, [4] * B, 4, 8, max_len, window=512) == want
            assert cluster(plan, [4] * B, 4, 8, max_len) >= want
    assert cluster(plan, [4, 4], 4, 1, 32768) == 8
    assert cluster(plan, [4, 4], 4, 1, 32768, window=512) <= 4


def test_choices(plan):
    """The measured cases, and batches behind wide tables that the GPU tests share by clusters of
    every size."""
    assert cluster(plan, [4, 4], 4, 8, 2048) == 4
    assert cluster(plan, [5] * 8, 4, 8, 4096) == 2
    assert cluster(plan, [512], 4, 8, 512) == 1
    assert cluster(plan, [2048], 8, 8, 32768) == 2
    assert cluster(plan, [2048], 8, 8, 8192) == 1
    assert cluster(plan, [2800] * 4, 4, 8, 131072) == 1
    new = (150, 20, 200, 90)
    for B, want in ((3, 8), (12, 4), (26, 2)):
        for us in (1.2, 1.5, 1.75):
            assert cluster(plan, [new[i % 4] for i in range(B)], 4, 1, 16 * 4096, us=us) == want
    for new in ((150, 20, 200), (3, 2, 1)):
        for us in (1.2, 1.5, 1.75):
            assert cluster(plan, new, 4, 1, 16 * 4096, window=1500, us=us) == 8
    assert cluster(plan, [3], 4, 1, 1 << 20, fit=(152, 0, 0, 0)) == 1
