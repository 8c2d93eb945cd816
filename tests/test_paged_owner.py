"""Which sequence each new row of a paged batch belongs to, on the host: by the definition where
query_start ascends, and never one whose rows it is not, or a malformed one, where it does not."""
from __future__ import annotations

import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def owners(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("owner") / "owner.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-x", "c++",
                    os.path.join(ROOT, "tests", "paged_owner_host.cpp"), "-I",
                    os.path.join(ROOT, "sliding_window_gqa_02_gb300", "csrc"), "-o", so], check=True)
    lib = ctypes.CDLL(so)

    def run(starts, lengths, N, max_new, max_len):
        q, k = np.array(starts, np.int32), np.array(lengths, np.int64).astype(np.int32) - 1
        out = np.full(N, -9, np.int32)
        at = lambda x: x.ctypes.data_as(ctypes.c_void_p)
        lib.paged_owners(at(q), at(k), len(lengths), N, max_new, max_len, N, at(out))
        return out.tolist()

    return run


def claims(starts, lengths, N, max_new, max_len):
    """For each row, the sequences that hold it and that the header does not call malformed."""
    out = [[] for _ in range(N)]
    for b, T in enumerate(lengths):
        q0, q1 = starts[b], starts[b + 1]
        if q0 < 0 or q1 < q0 or q1 > N or q1 - q0 > max_new or T < q1 - q0 or T > max_len:
            continue
        for n in range(q0, q1):
            out[n].append(b)
    return out


def check(owners, starts, lengths, N, max_new, max_len):
    got, want = owners(starts, lengths, N, max_new, max_len), claims(starts, lengths, N, max_new, max_len)
    for n in range(N):
        if want[n]:
            assert got[n] in want[n], (n, got[n], want[n])
        else:
            assert got[n] == -1, (n, got[n])


@pytest.mark.parametrize("starts,lengths,max_new", [
    ([0, 50, 60, 3, 108], [50, 20, 0, 200], 50),   # the last starts in the first's rows
    ([0, 50, 60, 3, 108], [50, 20, 0, 200], 108),  # ... and is well formed but for that
    ([0, 4, 8, 1, 9], [31, 11, 6, 21], 4),
    ([0, 6, 5, 6], [30, 40, 90], 3),
    ([10, 50, 3, 4], [60, 9, 9], 40),              # rows behind query_start[B] that are somebody's
    ([0, 0, 0, 7, 7], [0, 5, 7, 9], 7),
    ([-3, 2, 9], [8, 8], 9),
    ([3, 3, 300], [0, 4], 300),
    ([5], [], 0),
])
def test_listed(owners, starts, lengths, max_new):
    check(owners, starts, lengths, 110, max_new, 200)


@pytest.mark.parametrize("order", ["ascending", "one lower", "any"])
def test_random(owners, order):
    rng = random.Random(order)
    for _ in range(400):
        B = rng.choice([1, 2, 5, 31, 32, 33, 64, 65, 200, 1025])
        most = rng.choice([1, 3, 20])
        starts = [rng.choice([0, 0, 2])]
        for _ in range(B):
            starts.append(starts[-1] + rng.choice([0, 1, rng.randint(0, most)]))
        N = starts[-1] + rng.choice([0, 3])
        if order == "one lower" and B > 1:
            i = rng.randint(1, B)
            starts[i] = rng.randint(-1, starts[i])
        elif order == "any":
            starts = [rng.randint(-1, N + 1) for _ in starts]
        lengths = [rng.choice([0, 1, most, rng.randint(-2, 60), 1000]) for _ in range(B)]
        if rng.random() < 0.5:
            lengths = [starts[b + 1] - starts[b] + rng.randint(0, 5) for b in range(B)]
        check(owners, starts, lengths, N, rng.choice([most, N]), 500)
