"""Malformed sequences in a paged batch, on a GB300: flagged, not touched, and nothing else touched
for them.  The pages are compared bit for bit, rows that nobody appends to included."""
from __future__ import annotations

import pytest
import torch

from paged_driver import Batch
from sliding_window_gqa_02_gb300 import gqaw

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("at,length", [(1, 1000), (1, -2), (3, -1000), (70, 41), (3, 2 ** 31 - 1)])
@pytest.mark.parametrize("call", ["gqaw_paged_append", "gqaw_paged_attend", "gqaw_paged_step"])
def test_sequences_without_rows_are_flagged(call, at, length, dtype):
    """No row is theirs, so no row's warp can tell."""
    lens = [(2, 30), (0, 9), (3, 40), (0, 0)] + [(0, 5)] * 80
    b = Batch(lens, 4, 2, 64, 16, dtype, seed=31, filled=call == "gqaw_paged_attend")
    b.seqlens[at] = length
    k0, v0 = b.kp.clone(), b.vp.clone()
    b.call(getattr(gqaw, call), flags=gqaw.GQAW_DEV_BAD_SEQLEN)
    if call != "gqaw_paged_attend":
        b.check_pages(k0, v0)
    if call != "gqaw_paged_append":
        b.check_output()
