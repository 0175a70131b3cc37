"""Where the rows of a group lie (csrc/tfp8_groups.hpp), on the host: the header's code runs in a
wavefront of 64 coroutines (tests/wave_emulation) and is compared with the offsets' definition, for
offsets that keep the rules and for others."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def groups_lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("wave") / "groups.so")
    src = os.path.join(HERE, "wave_emulation")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", src, "-o", out,
                    os.path.join(src, "groups.cpp")], check=True)
    L = ctypes.CDLL(out)
    i64, p = ctypes.c_int64, ctypes.c_void_p
    L.tile.argtypes = [p, ctypes.c_int, i64, ctypes.c_int, ctypes.c_int, i64, p]
    L.span.argtypes = [p, ctypes.c_int, i64, ctypes.c_int, ctypes.c_int, p]
    return L


def call(f, off, *args):
    off = np.ascontiguousarray(off, np.int64)
    to = np.zeros(4, np.int64)
    assert f(off.ctypes.data, off.size - 1, *args, to.ctypes.data) == 0, "the lanes disagree"
    return to.tolist()


def parts_of(off, rows, all_rows):
    """(group, first row, end) of every group, and of the rows before the first and past the last."""
    at = np.maximum.accumulate(np.clip(np.asarray(off, np.int64), 0, rows)).tolist()
    parts = [(g, lo, hi) for g, (lo, hi) in enumerate(zip(at, at[1:]))]
    return [(-1, 0, at[0]), *parts, (-1, at[-1], rows)] if all_rows else parts


def tiles_of(off, rows, size, all_rows):
    return [(r, min(size, hi - r), g) for g, lo, hi in parts_of(off, rows, all_rows)
            for r in range(lo, hi, size)]


def offsets(counts, start=0):
    return np.concatenate([[0], np.cumsum(counts)]) + start


rng = np.random.default_rng(0)
CASES = {
    "even": (offsets([40] * 5), 200),
    "ragged": (offsets([7, 0, 130, 1, 300]), 438),
    "rows past the last": (offsets([20, 0, 33]), 100),
    "rows before the first": (offsets([20, 0, 33], 45), 98),
    "rows on both sides": (offsets([20, 0, 33], 5), 71),
    "empty": (offsets([0] * 7), 0),
    "no group has a row": (offsets([0] * 70, 30), 61),
    "63 groups": (offsets(rng.integers(0, 40, 63), 3), 1500),
    "64 groups": (offsets(rng.integers(0, 40, 64), 3), 1600),
    "65 groups": (offsets(rng.integers(0, 40, 65), 3), 1600),
    "200 groups": (offsets(rng.integers(0, 3, 200), 1), 400),
    "descending": ([90, 20, 80, 10], 100),
    "overlapping": ([0, 60, 30, 100, 10, 100], 100),
    "out of range": ([-9, 200, 50, 1 << 62], 100),
    "far out of range": ([0, -5, 1 << 40, 100], 100),
    "unsorted, 190 groups": (rng.integers(-10, 500, 191), 480),
    "sorted but one at the end of a wavefront": (np.r_[np.arange(0, 128, 2), 60, 130:260:2], 300),
    "all the same rows": (np.tile([0, 77], 40), 77),
}


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("size", [16, 128])
@pytest.mark.parametrize("all_rows", [True, False])
def test_tiles_hold_every_row_once(groups_lib, case, size, all_rows):
    off, rows = CASES[case]
    want = tiles_of(off, rows, size, all_rows)
    for i, w in enumerate(want):
        assert tuple(call(groups_lib.tile, off, rows, size, int(all_rows), i)) == (*w, len(want))
    assert call(groups_lib.tile, off, rows, size, int(all_rows), len(want))[1] == 0
    held = np.zeros(rows, int)
    for r, n, _ in want:
        held[r:r + n] += 1
    assert (held == 1).all() if all_rows else (held <= 1).all()
    # no more of them than a launch is for (both ends count as groups of their own)
    n = min(rows, len(off) + 1)
    assert len(want) <= (rows + n * (size - 1)) // size


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("size", [128, 512])
def test_spans_follow_the_tiles(groups_lib, case, size):
    off, rows = CASES[case]
    unit = 0
    for g, lo, hi in parts_of(off, rows, False):
        n = (hi - lo + size - 1) // size
        assert call(groups_lib.span, off, rows, size, g)[:2] == [unit, n]
        unit += n
    assert unit <= (rows + (len(off) - 1) * (size - 1)) // size


def test_sums_stay_in_range_with_most_rows(groups_lib):
    """2^31 - 1 rows: tiles of 16 of every group counted once, whatever the offsets claim."""
    rows = (1 << 31) - 1
    for off in (np.tile([0, rows], 40), np.tile([0, 1 << 62], 70), [0, rows // 3, rows]):
        want = sum((hi - lo + 15) // 16 for _, lo, hi in parts_of(off, rows, True))
        for i in (0, want // 2, want - 1):
            r, n, _, there = call(groups_lib.tile, off, rows, 16, 1, i)
            assert there == want and 0 <= r < rows and 0 < n <= 16 and r + n <= rows
        assert call(groups_lib.tile, off, rows, 16, 1, want)[1] == 0
