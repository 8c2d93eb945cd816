"""Sizes and strides whose products pass 64 bits, without a GPU: refused for what they are, and not
after wrapping into a size that looks right."""
from __future__ import annotations

import pytest

from test_paged_host import _paged, _qk, lib  # noqa: F401

T40 = 1 << 40
STRIDES = dict(page_stride=T40, head_stride=1 << 20, row_stride=64)


@pytest.mark.parametrize("over,msg", [
    # (2^28 + 1 - 1) pages of 2^40 elements are 2^68: 0 modulo 2^64
    (dict(STRIDES, num_pages=(1 << 28) + 1), "pages reach"),
    (dict(STRIDES, num_pages=1 << 9), "pages reach"),
    (dict(page_size=1 << 24, page_table_width=1, num_pages=1 << 30), "pages reach"),
    (dict(query_stride=T40, total_new_tokens=1 << 20), "query_stride"),
    (dict(key_stride=T40, total_new_tokens=(1 << 24) + 1), "key_stride"),
    (dict(value_stride=1 << 36, total_new_tokens=1 << 13), "value_stride"),
    (dict(output_stride=T40, total_new_tokens=(1 << 24) + 1), "output_stride"),
])
def test_paged(lib, over, msg):  # noqa: F811
    for fn in (lib.gqaw_paged_append, lib.gqaw_paged_attend, lib.gqaw_paged_step):
        assert fn(_paged(lib, **over), 0) == lib.GQAW_EUNSUPPORTED
        assert msg in lib.gqaw_last_error(), lib.gqaw_last_error()
    assert lib.gqaw_paged_workspace_bytes(_paged(lib, **over)) == 0


def test_rows_of_a_page_that_wrap(lib):  # noqa: F811
    """2^24 rows 2^40 elements apart are 2^64: a head stride above none of them."""
    a = _paged(lib, page_size=(1 << 24) + 1, row_stride=T40, head_stride=1 << 20, page_stride=T40)
    assert lib.gqaw_paged_append(a, 0) == lib.GQAW_EINVAL
    assert "overlap" in lib.gqaw_last_error()


@pytest.mark.parametrize("name", ["query_stride", "key_stride", "query_out_stride", "key_out_stride"])
def test_qk(lib, name):  # noqa: F811
    a = _qk(lib, **{name: T40, "num_tokens": (1 << 24) + 1})
    assert lib.gqaw_qk_norm_rotary(a, 0) == lib.GQAW_EUNSUPPORTED
    assert name in lib.gqaw_last_error()


def test_large_caches_that_fit_are_taken(lib):  # noqa: F811
    """256 GB of pages, and rows as far apart as a stride may be."""
    assert lib.gqaw_paged_workspace_bytes(_paged(lib, num_pages=1 << 24, page_size=32, kv_num_heads=4, page_table_width=7)) > 0
    assert lib.gqaw_paged_workspace_bytes(_paged(lib, query_stride=T40)) > 0
