"""Runs of row tiles (csrc/product_runs.h) against the kernel's mapping of workgroups to
row tiles, written out again here, with workgroup h on XCD h mod 8."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "align_moe_route_amd", "csrc")

SOURCE = """#include "product_runs.h"
extern "C" int runs(int64_t experts, int64_t average, int bm, int block) { return run_of(experts, average, bm, block); }
extern "C" bool fits(int64_t experts, int64_t average, int bm, int block, int64_t columns) {
  return at_once(experts, average, bm, block, columns);
}
"""


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("runs")
    (at / "runs.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-I", CSRC, str(at / "runs.cpp"), "-o",
                    str(at / "runs.so")], check=True)
    lib = ctypes.CDLL(str(at / "runs.so"))
    lib.runs.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    lib.fits.argtypes, lib.fits.restype = lib.runs.argtypes + [ctypes.c_int64], ctypes.c_bool
    return lib


@pytest.fixture
def run_of(library):
    return library.runs


@pytest.fixture
def at_once(library):
    return library.fits


def tiles_of_xcds(experts, average, bm, block, run):
    """Row tiles with a route on each XCD, and every tile that a workgroup takes."""
    blocks = -(-average // block)
    stride, live = blocks * (block // bm), -(-average // bm)
    tiles = experts * stride
    group = 8 << run
    of, taken = [0] * 8, []
    for h in range(-(-tiles // group) * group):
        x, i = h % 8, h // 8
        rt = (i >> run << 3 | x) << run | (i & ((1 << run) - 1))
        if rt < tiles:
            taken.append(rt)
            of[x] += rt % stride < live
    assert sorted(taken) == list(range(tiles))
    assert sum(of) == experts * live
    return of


SIZES = [  # experts, average rows, rows of a tile, block
    (1, 512, 64, 128), (4, 128, 64, 64), (8, 75, 64, 128), (8, 128, 64, 128), (2, 400, 64, 128), (1, 300, 64, 64),
    (64, 1, 64, 4096), (16, 8, 64, 1024), (16, 8, 128, 2048), (40, 3, 16, 4096), (8, 64, 128, 1024), (1, 1, 16, 16), (3, 40, 16, 48),
    (64, 64, 128, 128), (64, 256, 64, 64), (896, 147, 128, 128), (896, 2, 16, 16), (24, 195, 64, 64), (5, 205, 64, 128),
    (8, 1024, 128, 128), (1, 5000, 128, 4096), (100, 20, 32, 96), (7, 33, 16, 16)]


@pytest.mark.parametrize("experts,average,bm,block", SIZES)
def test_no_run_is_much_better(run_of, experts, average, bm, block):
    """Either every XCD has a tile, or no other run would halve the busiest one's."""
    of = tiles_of_xcds(experts, average, bm, block, run_of(experts, average, bm, block))
    if min(of) == 0:
        best = min(max(tiles_of_xcds(experts, average, bm, block, run)) for run in range(9))
        assert max(of) < 2 * best or max(of) == 1


@pytest.mark.parametrize("experts,average,bm,block", [(1, 512, 64, 128), (4, 128, 64, 64), (8, 75, 64, 128), (8, 128, 64, 128),
                                                      (64, 1, 64, 4096), (16, 8, 64, 1024)])
def test_every_xcd_has_a_tile(run_of, experts, average, bm, block):
    assert min(tiles_of_xcds(experts, average, bm, block, run_of(experts, average, bm, block))) > 0


@pytest.mark.parametrize("sizes,run", [((64, 64, 128, 128), 0), ((64, 256, 64, 64), 2), ((896, 147, 128, 128), 2),
                                       ((24, 195, 64, 64), 2), ((896, 2, 16, 16), 0), ((8, 1024, 128, 128), 2),
                                       ((5, 205, 64, 128), 2), ((896, 1, 64, 128), 1)])
def test_runs_share_an_experts_weights(run_of, sizes, run):
    """Where every XCD has tiles either way, or sharing is worth more."""
    assert run_of(*sizes) == run


def test_it_is_chosen_in_no_time(run_of):
    """Sizes at the ends of the range: the choice looks at a bounded number of runs."""
    import time
    worst = [(1, 2 ** 30, 16, 16), (1, 2 ** 26, 128, 4096), (4096, 2 ** 18, 128, 1 << 20), (4096, 1, 16, 1 << 30),
             (64, 2600, 64, 4096), (4096, 1, 16, 16)]
    for sizes in worst:
        run_of(*sizes)
        start = time.perf_counter()
        for _ in range(100):
            run_of(*sizes)
        assert time.perf_counter() - start < 0.05, sizes  # half a millisecond each


@pytest.mark.parametrize("sizes,columns,fits", [
    ((8, 75, 64, 128), 16, True), ((8, 100, 64, 128), 20, True), ((4, 100, 64, 128), 64, True), ((1, 512, 64, 128), 32, True),
    ((8, 128, 64, 128), 24, False),   # an expert of 128 rows on average has more than two tiles as often as not
    ((2, 1000, 64, 128), 16, False), ((5, 280, 64, 128), 20, False), ((1, 10 ** 6, 64, 128), 16, False)])
def test_narrow_tiles_at_once(at_once, sizes, columns, fits):
    assert at_once(*sizes, columns) == fits
