"""Paged steps over keys and values woven into one tensor at every level, on a GB300."""
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
@pytest.mark.parametrize("at", [0, 1, 2, 3])
@pytest.mark.parametrize("inside", [False, True], ids=["rows inside heads", "heads inside rows"])
@pytest.mark.parametrize("lens", [[(1, 40), (0, 3), (2, 200)], [(40, 300), (1, 70), (100, 100)]], ids=["decode", "chunks"])
def test_step(lens, inside, at, dtype):
    """at: where the dimension of (key, value) stands among pages, heads and rows."""
    b = Batch(lens, 8, 2, 64, 16, dtype, seed=51, heads_inside_rows=inside, norm=True, rotary=64, filled=False)
    k0, v0 = b.kp.clone(), b.vp.clone()
    both = torch.stack([b.kp, b.vp], at)
    b.kp, b.vp = both.select(at, 0), both.select(at, 1)
    assert b.kp.data_ptr() + both.stride(at) * both.element_size() == b.vp.data_ptr()
    b.call(gqaw.gqaw_paged_step)
    b.check_pages(k0, v0)
    b.check_output(turned=True, parts=2 if dtype == BF else 1)
    b.check_untouched()
