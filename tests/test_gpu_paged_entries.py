"""Page table entries out of range, whatever they are, in every attention kernel of the paged operators."""
from __future__ import annotations

import pytest
import torch

from paged_driver import Batch
from sliding_window_gqa_02_gb300 import gqaw

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("entry", [-1, -2, -3, -(1 << 31), 1 << 20, (1 << 31) - 1])
@pytest.mark.parametrize("dtype,S,Nq,D,page", [
    (BF, 1, 4, 64, 16), (BF, 1, 4, 256, 32), (BF, 40, 4, 128, 16), (BF, 200, 4, 64, 128), (BF, 70, 4, 256, 64),  # tensor cores
    (F, 1, 4, 64, 16), (F, 2, 4, 128, 32),   # fp32 decode by tensor copies
    (F, 1, 4, 32, 7), (F, 3, 2, 128, 5), (F, 4, 2, 256, 16),  # a warp a tile
    (F, 40, 4, 64, 16), (BF, 3, 4, 32, 16), (BF, 5, 4, 64, 12), (F, 9, 8, 16, 3)])  # by rows
def test_every_bad_entry_is_flagged(entry, dtype, S, Nq, D, page):
    t = Batch([(S, 310), (S, 200), (1, 33)], Nq, 2, D, page, dtype, seed=61, window=250)
    t.table[0, max(0, 310 - S - 250 + 1) // page + 1] = entry
    t.call(gqaw.gqaw_paged_attend, flags=gqaw.GQAW_DEV_BAD_PAGE)
    t.check_output(skip=(0,))
    u = Batch([(S, 110 + S + page), (1, 40)], Nq, 2, D, page, dtype, seed=62, window=20)
    u.table[0, 0] = entry
    u.call(gqaw.gqaw_paged_attend)
    u.check_output()
