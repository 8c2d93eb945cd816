"""Keys and values of a paged cache woven into one tensor, without a GPU: every layout in which no
two rows share an element is let through to the device checks, every other one refused."""
from __future__ import annotations

import itertools

import pytest

from test_paged_host import _paged, lib  # noqa: F401

BASE = 1 << 34


def _strides(order, sizes, D, at):
    """Strides (elements) of a tensor whose dimensions are `order`, innermost last, then D; `kv` has 2."""
    out, step = {}, D
    for name in reversed(order):
        out[name] = step
        step *= sizes[name]
    return out


ORDERS = [o for n in range(4) for base in (("page", "head", "row"), ("page", "row", "head"))
          for o in [base[:n] + ("kv",) + base[n:]]]


def _call(lib, gap, st, sizes, fn):  # noqa: F811
    a = _paged(lib, key_pages=BASE, value_pages=BASE + gap * 2, page_stride=st["page"], head_stride=st["head"],
               row_stride=st["row"], num_pages=sizes["page"], kv_num_heads=sizes["head"], page_size=sizes["row"],
               num_heads=sizes["head"], head_size=16, page_table_width=200, max_sequence_length=100)
    got = getattr(lib, fn)(a, 0)
    assert got != lib.GQAW_OK  # the addresses are not a device's
    return "overlaps" in lib.gqaw_last_error()


@pytest.mark.parametrize("fn", ["gqaw_paged_append", "gqaw_paged_step"])
@pytest.mark.parametrize("sizes", [(5, 2, 8), (1, 4, 8), (3, 1, 8), (4, 3, 1), (1, 1, 2), (1, 1, 1)], ids=str)
@pytest.mark.parametrize("order", ORDERS, ids="-".join)
def test_layouts(lib, order, sizes, fn):  # noqa: F811
    sizes = dict(zip(("page", "head", "row"), sizes), kv=2)
    st = _strides(order, sizes, 16, None)
    assert not _call(lib, st["kv"], st, sizes, fn)
    assert not _call(lib, -st["kv"], st, sizes, fn)


@pytest.mark.parametrize("order", ORDERS, ids="-".join)
def test_gaps(lib, order):  # noqa: F811
    """Any gap: refused exactly if some key row and some value row share an element, but for
    tensors that interleave in a way that is not one level's blocks, which are refused too."""
    sizes = dict(page=3, head=2, row=4, kv=2)
    st = _strides(order, sizes, 16, None)
    rows = {p * st["page"] + h * st["head"] + r * st["row"]
            for p, h, r in itertools.product(range(3), range(2), range(4))}
    span = max(rows) + 16
    allowed = 0
    for gap in range(-span - 16, span + 17, 8):
        share = any(abs(x - y - gap) < 16 for x in rows for y in rows)
        refused = _call(lib, gap, st, sizes, "gqaw_paged_append")
        assert refused or not share, gap
        allowed += not refused
        if abs(gap) == st["kv"] or abs(gap) >= span:
            assert not refused, gap
    assert allowed
