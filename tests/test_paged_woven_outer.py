"""Keys and values of a paged cache woven into one tensor whose outer strides step over one of them alone, without a GPU."""
from __future__ import annotations

import itertools
import random

import pytest

from test_paged_host import _paged, lib  # noqa: F401
from test_paged_woven import _call

D = 16


def test_an_outer_stride_that_steps_over_the_keys_alone(lib):  # noqa: F811
    """The next head, or page, begins where the keys end: on the last row of values."""
    sizes = dict(page=3, head=2, row=8)
    keys = 7 * 2 * D + D  # what a head's keys reach over
    assert _call(lib, D, dict(row=2 * D, head=keys, page=1 << 12), sizes, "gqaw_paged_append")
    assert not _call(lib, D, dict(row=2 * D, head=keys + D, page=1 << 12), sizes, "gqaw_paged_append")
    sizes = dict(page=3, head=1, row=8)
    assert _call(lib, D, dict(row=2 * D, head=keys, page=keys), sizes, "gqaw_paged_append")
    assert not _call(lib, D, dict(row=2 * D, head=keys, page=keys + D), sizes, "gqaw_paged_append")


@pytest.mark.parametrize("seed", range(4))
def test_no_overlap_is_let_through(lib, seed):  # noqa: F811
    rng = random.Random(seed)
    let = 0
    for _ in range(1500):
        sizes = dict(page=rng.choice([1, 2, 3]), head=rng.choice([1, 2, 3]), row=rng.choice([1, 2, 4]))
        a, b = rng.choice([("row", "head"), ("head", "row")])
        st = {a: D * rng.choice([1, 2, 3])}
        st[b] = max(D, (sizes[a] - 1) * st[a] + D) + D * rng.choice([0, 0, 1, 2, 5])
        st["page"] = (sizes[b] - 1) * st[b] + (sizes[a] - 1) * st[a] + D + D * rng.choice([0, 0, 1, 2, 9])
        gap = D * rng.randint(-20, 20) + rng.choice([0, 0, 8])
        rows = {p * st["page"] + h * st["head"] + r * st["row"]
                for p, h, r in itertools.product(range(sizes["page"]), range(sizes["head"]), range(sizes["row"]))}
        share = any(abs(x - y - gap) < D for x in rows for y in rows)
        refused = _call(lib, gap, st, sizes, "gqaw_paged_append")
        assert refused or not share, (sizes, st, gap)
        let += not refused
    assert let > 50
