"""Parts of a 4-bit cache woven into one buffer, on the host: a call is refused where two of the bytes that it may write
are one, and no layout is let through that brute force finds overlapping."""
from __future__ import annotations

import random

import numpy as np
import pytest

from test_i4_host import _args, _reaches_device, lib  # noqa: F401 (a fixture)

BASE = 1 << 33


def rows(page, head, row, n, heads, size):
    """The first bytes of all rows of a part."""
    i = np.arange
    return (i(n)[:, None, None] * page + i(heads)[None, :, None] * head + i(size)[None, None, :] * row).ravel()


def overlapping(parts):
    """parts: (offset, page, head, row strides in bytes, bytes of a row), of the same numbers of pages, heads and rows."""
    start, end = [], []
    for at, page, head, row, width, n, heads, size in parts:
        r = at + rows(page, head, row, n, heads, size)
        start.append(r)
        end.append(r + width)
    start, end = np.concatenate(start), np.concatenate(end)
    order = np.argsort(start, kind="stable")
    return bool((end[order][:-1] > start[order][1:]).any())


def layout(lib, D, n, heads, size, codes, scales, at):
    """Arguments of an append whose four parts lie at `at` with strides `codes` and `scales` in bytes."""
    return dict(head_size=D, num_heads=heads, kv_num_heads=heads, page_size=size, num_pages=n, page_table_width=1, max_sequence_length=size,
                max_new_tokens=1, total_new_tokens=1, batch_size=1,
                page_stride=codes[0], head_stride=codes[1], row_stride=codes[2],
                scale_page_stride=scales[0] // 2, scale_head_stride=scales[1] // 2, scale_row_stride=scales[2] // 2,
                key_pages=BASE + at[0], value_pages=BASE + at[1], key_scales=BASE + at[2], value_scales=BASE + at[3])


def test_an_outer_stride_that_steps_over_one_part_alone(lib):  # noqa: F811
    """Keys and values row by row, and the next head (or page) where the keys end: the last row of values is the next
    one's first row of keys."""
    D, size = 64, 16
    w, s = D // 2, D // 32 * 2
    head = (size - 1) * 2 * w + w  # what the keys of a head reach over
    far = 1 << 24
    args = layout(lib, D, 3, 4, size, (1 << 16, head, 2 * w), (1 << 12, size * s, s), (0, w, far, 2 * far))
    assert lib.gqaw_paged_i4_append(_args(lib, **args), 0) == lib.GQAW_EINVAL
    assert "key_pages overlaps value_pages" in lib.gqaw_last_error()
    args = layout(lib, D, 3, 1, size, (head, head, 2 * w), (1 << 12, size * s, s), (0, w, far, 2 * far))
    assert lib.gqaw_paged_i4_append(_args(lib, **args), 0) == lib.GQAW_EINVAL
    good = layout(lib, D, 3, 4, size, (1 << 16, head + w, 2 * w), (1 << 12, size * s, s), (0, w, far, 2 * far))
    assert _reaches_device(lib, "gqaw_paged_i4_append", **good), lib.gqaw_last_error()


@pytest.mark.parametrize("seed", range(4))
def test_no_overlap_is_let_through(lib, seed):  # noqa: F811
    rng = random.Random(seed)
    let, refused = 0, 0
    for _ in range(4000):
        D = rng.choice([32, 64, 128])
        w, s = D // 2, D // 32 * 2
        n, heads, size = rng.choice([1, 2, 3]), rng.choice([1, 2, 3]), rng.choice([1, 2, 4])

        def strides(width, unit):
            up = lambda x: -(-x // unit) * unit  # noqa: E731
            inner = up(width) * rng.choice([1, 1, 2, 4])
            if rng.random() < 0.5:  # rows inside heads
                row = inner
                head = up(max(width, (size - 1) * row + width)) + rng.choice([0, 0, 1, 2, 4]) * up(width)
                page = (heads - 1) * head + (size - 1) * row + width
            else:
                head = inner
                row = up(max(width, (heads - 1) * head + width)) + rng.choice([0, 0, 1, 2, 4]) * up(width)
                page = (size - 1) * row + (heads - 1) * head + width
            return up(page) + rng.choice([0, 0, 1, 2, 8]) * up(width), head, row

        codes, scales = strides(w, 16), strides(s, max(s, 2))
        at = [0] + [rng.choice([16, 32, 64, 128, 256, 512]) * rng.randint(0, 9) for _ in "123"]
        args = layout(lib, D, n, heads, size, codes, scales, at)
        over = overlapping([(at[k], *(codes if k < 2 else scales), w if k < 2 else s, n, heads, size) for k in range(4)])
        st = lib.gqaw_paged_i4_append(_args(lib, **args), 0)
        if st == lib.GQAW_EINVAL and "overlap" in lib.gqaw_last_error():
            refused += 1
        else:
            assert st == lib.GQAW_ECUDA or "device" in lib.gqaw_last_error(), lib.gqaw_last_error()
            assert not over, (args, lib.gqaw_last_error())
            let += 1
    assert let > 50 and refused > 500
