"""What the binding of the paged operators refuses before the library sees it (CPU tensors: nothing
is called with them)."""
from __future__ import annotations

import pytest
import torch

from test_paged_host import lib  # noqa: F401


@pytest.mark.parametrize("shape", [(9, 0), (0, 32), (0, 0)])
def test_empty_tables(lib, shape):  # noqa: F811
    """A tensor without elements has no address: the call would turn nothing, and say nothing."""
    rows, kv, pages = torch.zeros(5, 4 * 64), torch.zeros(5, 2 * 64), torch.zeros(3, 2, 8, 64)
    table, start, lens = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ids = torch.zeros(5, dtype=torch.int64)
    for cos, sin in ((torch.zeros(shape), torch.zeros(shape)), (torch.zeros(9, 32)[:shape[0], :shape[1]],) * 2):
        with pytest.raises(ValueError, match="cos_cache"):
            lib.make_paged_args(rows, kv, kv, pages, pages, table, start, lens, 5, 24, 4, 2, rows, cos_cache=cos, sin_cache=sin)
        with pytest.raises(ValueError, match="cos_cache"):
            lib.make_qk_args(rows, None, rows, None, 4, 0, 64, cos_cache=cos, sin_cache=sin, position_ids=ids)
    t = torch.zeros(9, 32)
    assert lib.make_qk_args(rows, None, rows, None, 4, 0, 64, cos_cache=t, sin_cache=t, position_ids=ids).rotary_dim == 64
