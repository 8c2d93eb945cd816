"""The schedule of the paged attention, on the host: every key tile of every unit is taken by
exactly one CTA, the tiles are the ones the mask needs, and what the merge relies on holds."""
from __future__ import annotations

import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sched(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("sched") / "sched.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-x", "c++",
                    os.path.join(ROOT, "tests", "paged_sched_host.cpp"), "-I",
                    os.path.join(ROOT, "sliding_window_gqa_02_gb300", "csrc"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.paged_schedule.restype = ctypes.c_longlong

    def run(lens, tpt, window, heads, grid, keys, cost):
        flat = np.array([x for st in lens for x in st], np.int32)
        cap = 200000
        out, tot = np.zeros((cap, 12), np.int64), np.zeros(3, np.int64)
        n = lib.paged_schedule(flat.ctypes.data_as(ctypes.c_void_p), len(lens), tpt, window, heads, grid, int(keys == 32), cost,
                               out.ctypes.data_as(ctypes.c_void_p), ctypes.c_longlong(cap),
                               tot.ctypes.data_as(ctypes.c_void_p))
        assert n >= 0
        return out[:n], tot

    return run


def check(run, lens, tpt, window, heads, grid, keys, cost):
    rows, tot = run(lens, tpt, window, heads, grid, keys, cost)
    want = {}
    row = 0
    for b, (S, T) in enumerate(lens):
        P = T - S
        for r in range((S + tpt - 1) // tpt):
            s0, s1 = r * tpt, min(S, (r + 1) * tpt)
            lo = max(0, P + s0 - window + 1) // keys if window else 0
            hi = (P + s1 - 1) // keys + 1
            for h in range(heads):
                want[(b, h, row + s0)] = (s1 - s0, P + s0, lo, hi - lo)
        row += S
    assert tot[1] == len(want) and tot[0] == sum(w[3] + cost for w in want.values())
    got, load = {}, {}
    for cta, b, hu, row0, ntok, qpos, kt, nt, k0, k1, cf, cl in rows.tolist():
        key = (b, hu, row0)
        assert want[key] == (ntok, qpos, kt, nt), (key, want[key], (ntok, qpos, kt, nt))
        assert 0 <= k0 < k1 <= nt
        got.setdefault(key, []).append((k0, k1, cta, cf, cl))
        load[cta] = load.get(cta, 0) + k1 - k0 + (cost if k0 == 0 else 0)
    assert set(got) == set(want)
    tickets = {}
    slots = set()
    for key, parts in got.items():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == want[key][3]
        assert all(x[1] == y[0] for x, y in zip(parts, parts[1:]))
        if len(parts) > 1:
            cf, cl = parts[0][3], parts[0][4]
            assert all(p[3] == cf and p[4] == cl for p in parts)
            assert [p[2] for p in parts] == list(range(cf, cl + 1))  # one part in each of cf .. cl
            assert cf not in tickets and 0 <= cf and cl < grid
            tickets[cf] = key
            for p in parts:  # the place of a CTA's partial result is its own
                slot = (p[2], p[2] == cf)
                assert slot not in slots
                slots.add(slot)
    return load, tot


CASES = [
    ([(8, 9000), (3, 16000)], 8, 0, 1, 152, 128),
    ([(8, 16000)] * 16, 8, 0, 8, 152, 128),
    ([(1, 131)], 1, 0, 8, 16, 128),
    ([(1, 32768)], 1, 0, 8, 152, 128),
    ([(2048, 2048), (77, 1077)], 32, 0, 8, 152, 128),
    ([(512, t) for t in (4608, 9000, 32768)], 32, 4096, 8, 152, 128),
    ([(0, 0), (5, 5), (0, 9), (1, 1)], 18, 0, 4, 152, 128),
    ([(129, 129)], 18, 7, 3, 608, 32),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_listed(sched, case):
    for cost in (0, 3):
        check(sched, *case, cost)


def test_random(sched):
    rng = random.Random(5)
    for _ in range(400):
        n = rng.randint(1, 60)
        top = rng.choice([3, 40, 300, 5000, 40000])
        most = rng.choice([1, 4, 40, 700])
        lens = []
        for _ in range(n):
            T = rng.randint(0, top)
            lens.append((min(T, rng.choice([0, 1, rng.randint(0, most)])), T))
        tpt = rng.choice([1, 2, 4, 8, 16, 18, 32, 42, 128])
        window = rng.choice([0, 0, 1, 5, 100, 128, 129, 3000, 4096])
        cost = rng.choice([0, 2, 3])
        load, tot = check(sched, lens, tpt, window, rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 16, 152, 608]),
                          rng.choice([32, 128]), cost)
        if load and not tot[2]:  # equal shares, but for a boundary inside a unit's fixed part
            assert max(load.values()) - min(load.values()) <= 1 + 2 * cost
