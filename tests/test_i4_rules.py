"""Rules of the operators on 4-bit caches, on the host."""
from __future__ import annotations

import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sliding_window_gqa_02_gb300", "csrc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rules") / "rules.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-x", "c++", os.path.join(ROOT, "tests", "i4_rules_host.cpp"),
                    "-I", CSRC, "-o", so], check=True)
    x = ctypes.CDLL(so)
    x.i4_blocks.argtypes = [ctypes.c_longlong] * 4
    x.i4_offsets_fit.argtypes = [ctypes.c_longlong] * 3
    return x


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_blocks_only_where_their_offsets_fit_32_bits(lib, D):
    rows, row, group = 1024 // D, D // 2, D // 32
    rng = random.Random(D)
    strides = [1 << n for n in range(9, 36)] + [rng.randrange(row, 1 << 36) for _ in range(300)]
    strides += [(1 << 32) // (rows - 1) + d for d in range(-64, 65, 16)]
    taken = 0
    for x in strides:
        sr, tr = max(row, x // 16 * 16), max(group, x // group * group)
        for a, b in ((sr, group), (row, tr), (sr, tr)):
            if lib.i4_blocks(rows * 2, D, a, b):
                taken += 1
                assert lib.i4_offsets_fit(D, a, b), (a, b)
            else:  # a fit is given up at the border alone
                assert not lib.i4_offsets_fit(D, a, b) or (rows - 1) * a + row > 1 << 32 or (rows - 1) * b >= 1 << 32
    assert taken
    # the usual layouts: a row's own bytes, heads inside rows, all four parts of a page in one buffer
    for heads in (1, 8, 128):
        assert lib.i4_blocks(rows, D, row * heads, group * heads) and lib.i4_blocks(rows * 4, D, 4096 * heads, 2048 * heads)
    assert not lib.i4_blocks(rows - 1, D, row, group) and not lib.i4_blocks(rows + 1, D, row, group)
    assert not lib.i4_blocks(rows, D, (1 << 32) // (rows - 1) // 16 * 16 + 16, group)
