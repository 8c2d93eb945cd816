"""The schedule of the paged attention with the tile widths, unit costs, tokens per tile and grids of
its kernels, on the host, and the warp's search 32 places at a time."""
from __future__ import annotations

import ctypes
import os
import random
import re
import subprocess

import numpy as np
import pytest

from test_paged_sched import check

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sliding_window_gqa_02_gb300", "csrc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("sched") / "sched.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-x", "c++",
                    os.path.join(ROOT, "tests", "paged_sched_kernels_host.cpp"), "-I", CSRC, "-o", so], check=True)
    x = ctypes.CDLL(so)
    x.paged_schedule_of.restype = ctypes.c_longlong
    return x


@pytest.fixture(scope="module")
def sched(lib):
    def run(lens, tpt, window, heads, grid, keys, cost):
        flat = np.array([x for st in lens for x in st], np.int32)
        cap = 400000
        out, tot = np.zeros((cap, 12), np.int64), np.zeros(3, np.int64)
        n = lib.paged_schedule_of(flat.ctypes.data_as(ctypes.c_void_p), len(lens), tpt, window, heads, grid, keys, cost,
                                  out.ctypes.data_as(ctypes.c_void_p), ctypes.c_longlong(cap),
                                  tot.ctypes.data_as(ctypes.c_void_p))
        assert n >= 0
        return out[:n], tot

    return run


# file, key tile, unit cost, tokens per query tile, grids
KERNELS = {
    "decode": ("gqaw_paged_dec.cu", 128, 2, [1, 2, 4, 8], [1, 9, 152]),
    "prompt": ("gqaw_paged_pre.cu", 128, 3, [1, 16, 18, 32, 42, 64, 128, 256], [152]),
    "fp32 decode": ("gqaw_paged_f32.cu", 16, 24, [1, 2, 4, 8], [152]),
    "a warp a tile": ("gqaw_paged_attend.cuh", 32, 4, [1, 2, 4, 8], [152, 304]),
    "rows": ("gqaw_paged_attend.cuh", 32, 4, [1, 2, 16, 18, 32, 128], [152, 608]),
}


@pytest.mark.parametrize("name", KERNELS)
def test_costs_are_those_of_the_kernels(name):
    src = open(os.path.join(CSRC, KERNELS[name][0])).read()
    assert int(re.search(r"constexpr int kUnitCost = (\d+);", src).group(1)) == KERNELS[name][2]


@pytest.mark.parametrize("name", KERNELS)
def test_random(sched, name):
    _, keys, cost, tpts, grids = KERNELS[name]
    rng = random.Random(name)
    for _ in range(300):
        tpt = rng.choice(tpts)
        top = rng.choice([3, 40, 300, 5000, 40000])
        few = name in ("decode", "fp32 decode", "a warp a tile")
        lens = []
        for _ in range(rng.choice([1, 2, 5, 30, 60, 256])):
            T = rng.randint(0, top)
            lens.append((min(T, rng.choice([0, 1, rng.randint(0, tpt if few else rng.choice([40, 700]))])), T))
        window = rng.choice([0, 0, 1, 5, 15, 16, 17, 100, 128, 129, 3000, 4096])
        load, tot = check(sched, lens, tpt, window, rng.choice([1, 2, 3, 8]), rng.choice(grids), keys, cost)
        if load and not tot[2]:  # equal shares, but for a boundary inside a unit's fixed part
            assert max(load.values()) - min(load.values()) <= 1 + 2 * cost


def test_search(lib):
    """The search by a warp's votes finds what going through the places finds."""
    for n in list(range(1, 200)) + [255, 256, 1023, 1024, 1025, 32768, 100001, 1 << 30]:
        for last in {0, 1, 2, 30, 31, 32, 33, n // 2, n - 2, n - 1}:
            if 0 <= last < n:
                assert lib.paged_last_where(n, last) == last, (n, last)
