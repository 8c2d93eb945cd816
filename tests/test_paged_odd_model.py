"""A model of how the prompt kernels hand over the bits of values that are not finite (no GPU).

In csrc/gqaw_paged_pre.cu the softmax warps of a CTA go through its units, each at its own pace
between barriers.  In unit i a warp sets bits in buffer i % n as it meets such values; then all
warps meet at a barrier, every warp reads the unit's bits at some time of its epilogue, and warp 0
clears buffer (i - 1) % n.  Nothing else orders the warps.  Every unit's bits must reach every warp,
and none of another unit's.  The model runs the warps under a random scheduler that likes to let one
warp run on; the number of buffers is read from the source.
"""
from __future__ import annotations

import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _buffers():
    src = open(os.path.join(ROOT, "sliding_window_gqa_02_gb300", "csrc", "gqaw_paged_pre.cu")).read()
    n = re.search(r"constexpr int kOddBufs = (\d+);", src)
    return int(n.group(1)) if n else 2  # without the constant: two, by the unit's parity


def _errors(n, seed, warps=4, units=8):
    rnd = random.Random(seed)
    buf = [set() for _ in range(n)]
    sets = [[{(i, w)} if rnd.random() < 0.5 else set() for w in range(warps)] for i in range(units)]
    met = [0] * units
    errors = []

    def warp(w):
        for i in range(units):
            yield
            buf[i % n].update(sets[i][w])
            yield
            met[i] += 1
            while met[i] < warps:
                yield
            if w == 0:
                first = rnd.random() < 0.5  # the clear before or after this warp's own reads
                if first:
                    buf[(i + n - 1) % n].clear()
                yield
            got = set(buf[i % n])
            if got != set().union(*sets[i]):
                errors.append("warp %d, unit %d: %s instead of %s" % (w, i, got, set().union(*sets[i])))
            yield
            if w == 0 and not first:
                buf[(i + n - 1) % n].clear()

    running = [warp(w) for w in range(warps)]
    weight = [rnd.choice([1, 1, 20]) for _ in running]
    while running:
        k = rnd.choices(range(len(running)), weight[:len(running)])[0]
        try:
            next(running[k])
        except StopIteration:
            running.pop(k)
            weight.pop(k)
    return errors


def test_bits_reach_every_warp_and_no_other_unit():
    for seed in range(2000):
        assert not _errors(_buffers(), seed), seed


@pytest.mark.parametrize("n", [2])
def test_the_model_sees_a_buffer_cleared_too_late(n):
    assert any(_errors(n, seed) for seed in range(200))
