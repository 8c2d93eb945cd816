"""The schedule of the attention over 4-bit caches on the host: every key tile of every unit is taken by exactly
one CTA, with the costs that the kernel has."""
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


def constants():
    src = open(os.path.join(CSRC, "gqaw_i4_attend.cuh")).read()
    names = ("kKeys", "kUnitCost", "kMergeCost", "kMinTiles")
    return {n: int(re.search(r"\b%s = (\d+)[,;]" % n, src).group(1)) for n in names}


@pytest.fixture(scope="module")
def sched(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("sched") / "i4.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-x", "c++",
                    os.path.join(ROOT, "tests", "i4_sched_host.cpp"), "-I", CSRC, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.i4_schedule.restype = ctypes.c_longlong
    c = constants()

    def run(lens, tpt, window, heads, grid, keys, cost):
        flat = np.array([x for st in lens for x in st], np.int32)
        cap = 400000
        out, tot = np.zeros((cap, 12), np.int64), np.zeros(3, np.int64)
        n = lib.i4_schedule(flat.ctypes.data_as(ctypes.c_void_p), len(lens), tpt, window, heads, grid, keys, cost,
                            c["kMergeCost"], c["kMinTiles"], out.ctypes.data_as(ctypes.c_void_p), ctypes.c_longlong(cap),
                            tot.ctypes.data_as(ctypes.c_void_p))
        assert n >= 0
        return out[:n], tot

    return run


@pytest.mark.parametrize("tpts", [[1, 2, 4, 8], [1, 3, 5, 16]])
@pytest.mark.parametrize("seed", [0, 1])
def test_random(sched, tpts, seed):
    c = constants()
    rng = random.Random(seed)
    for _ in range(150):
        tpt = rng.choice(tpts)
        top = rng.choice([3, 40, 300, 5000, 40000])
        lens = []
        for _ in range(rng.choice([1, 2, 5, 30, 60, 256])):
            T = rng.randint(0, top)
            lens.append((min(T, rng.choice([0, 1, rng.randint(0, rng.choice([tpt, 40, 300]))])), T))
        window = rng.choice([0, 0, 1, 5, 31, 32, 33, 100, 4096])
        load, tot = check(sched, lens, tpt, window, rng.choice([1, 2, 3, 8]), 152, c["kKeys"], c["kUnitCost"])
        if load and not tot[2]:  # equal shares, but for a boundary inside a unit's fixed part
            assert max(load.values()) - min(load.values()) <= 1 + 2 * c["kUnitCost"]


def test_long_units_are_cut_and_many_short_ones_are_not(sched):
    c = constants()
    _, tot = sched([(1, 100000)], 1, 0, 1, 152, c["kKeys"], c["kUnitCost"])
    assert not tot[2]
    rows, tot = sched([(1, 300)] * 50, 1, 0, 3, 152, c["kKeys"], c["kUnitCost"])
    assert tot[2] and len(rows) == 150
