"""Operators on 4-bit caches over layouts and tables that lie at the ends of what a call may give."""
from __future__ import annotations

import pytest
import torch

from i4_driver import Batch
from sliding_window_gqa_02_gb300 import gqaw

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
LONG = 1 << 20  # a length for which the expanded pages of a few sequences would be too large


@pytest.mark.parametrize("dtype,S", [(BF16, 1), (BF16, 3), (F32, 4)])
@pytest.mark.parametrize("D,row", [(32, 160 << 20), (64, 300 << 20), (128, 640 << 20), (256, 1500 << 20)])
def test_rows_far_apart(dtype, S, D, row):
    """Rows of a page so far apart that their offsets in a block of one copy pass 32 bits: codes, then scales."""
    page = 1024 // D
    for codes, scales in ((row, 0), (0, min(row, (1 << 32) // page * (D // 32) - 16))):  # a page of scales has an end of its own
        t = Batch([(S, page), (1, page - 1)], 4, 2, D, page, dtype, seed=41, norm=True, rotary=32, heads_inside_rows=True, spare_pages=0)
        far = []
        for x, stride in ((t.kc, codes), (t.vc, codes), (t.ks, scales), (t.vs, scales)):
            if stride:
                n, r = x.shape[:2]
                buf = torch.empty((n * r - 1) * stride + x[0, 0].numel(), dtype=x.dtype, device=x.device)
                y = buf.as_strided(x.shape, (r * stride, stride, *x.stride()[2:]))
                y.copy_(x)
                x = y
            far.append(x)
        t.kc, t.vc, t.ks, t.vs = far
        before = t.snapshot()
        t.call(gqaw.gqaw_paged_i4_step)
        t.check_pages(before)
        t.check_output(turned=True)
        t.call(gqaw.gqaw_paged_i4_read)
        t.check_read()
        del t, far, x, y, buf
        torch.cuda.empty_cache()


@pytest.mark.parametrize("entry", [-1, -2, -3, -(1 << 31), 1 << 20, (1 << 31) - 1])
@pytest.mark.parametrize("dtype,S,D,page,max_len", [(BF16, 1, 64, 16, 0), (BF16, 4, 128, 24, 0), (BF16, 2, 32, 16, 0), (F32, 3, 64, 16, 0),
                                                    (F32, 9, 128, 7, 0), (BF16, 100, 128, 16, 0), (BF16, 70, 64, 24, LONG),
                                                    (BF16, 60, 128, 16, LONG), (BF16, 90, 256, 32, 0)])
def test_every_bad_entry_is_flagged(entry, dtype, S, D, page, max_len):
    """A table entry out of range sets the flag, whatever it is, in every kernel; other sequences are right, and
    an entry that nobody needs is not looked at."""
    t = Batch([(S, 310), (S, 200), (1, 33), (S, 128)], 8, 2, D, page, dtype, seed=51, max_len=max_len, window=150)
    t.table[0, max(0, 310 - S - 150 + 1) // page + 2] = entry
    t.call(gqaw.gqaw_paged_i4_attend, flags=gqaw.GQAW_DEV_BAD_PAGE)
    t.check_output(skip=(0,))
    u = Batch([(S, 310), (1, 40)], 8, 2, D, page, dtype, seed=52, max_len=max_len, window=20)
    u.table[0, 0] = entry
    u.call(gqaw.gqaw_paged_i4_attend)
    u.check_output()


@pytest.mark.parametrize("dtype,S,D,max_len", [(BF16, 1, 64, 0), (BF16, 5, 32, 0), (F32, 3, 128, 0), (BF16, 1, 256, 0), (BF16, 100, 128, 0),
                                               (BF16, 90, 256, 0), (BF16, 60, 128, LONG)])
@pytest.mark.parametrize("page", [16, 1 << 22])
def test_a_cache_without_pages(dtype, S, D, max_len, page):
    """No page exists: every table entry is out of range, the tokens' outputs are unspecified, rows read back are left
    as they were.  With pages so large that a head's place lies beyond any memory of the call."""
    t = Batch([(S, 140), (0, 5), (1, 9), (S, 200)], 8, 2, D, 16, dtype, seed=53, norm=True, rotary=32, extra_rows=2, max_len=max_len)
    t.page = page
    t.kc, t.vc = (torch.empty(0, 2, page, D // 2, dtype=torch.uint8, device="cuda") for _ in "kv")
    t.ks, t.vs = (torch.empty(0, 2, page, D // 32, dtype=BF16, device="cuda") for _ in "kv")
    t.max_len = min(t.max_len, t.table.shape[1] * page)
    assert t.args().paged.num_pages == 0
    for call in (gqaw.gqaw_paged_i4_append, gqaw.gqaw_paged_i4_attend, gqaw.gqaw_paged_i4_step, gqaw.gqaw_paged_i4_read):
        t.call(call, flags=gqaw.GQAW_DEV_BAD_PAGE)
    assert (t.out[2 * S + 1:] == 7.0).all() and (t.ko == 7.0).all() and (t.vo == 7.0).all()


@pytest.mark.parametrize("dtype,max_new,D,max_len", [(BF16, 1, 64, 0), (BF16, 8, 128, 0), (F32, 20, 64, 0), (BF16, 300, 128, 0),
                                                     (BF16, 300, 256, 0), (BF16, 60, 128, LONG), (BF16, 60, 64, 4 * LONG)])
def test_a_batch_without_tokens(dtype, max_new, D, max_len):
    """Every sequence idle, though the call allows new tokens: the kernels run and find nothing to do."""
    t = Batch([(0, 90), (0, 0), (0, 400)], 8, 2, D, 16, dtype, seed=54, norm=True, rotary=32, extra_rows=max_new, max_len=max_len)
    t.max_new, t.max_len = max_new, max(t.max_len, max_new)
    before, launches = t.snapshot(), gqaw.gqaw_launch_count()
    for call in (gqaw.gqaw_paged_i4_append, gqaw.gqaw_paged_i4_attend, gqaw.gqaw_paged_i4_step, gqaw.gqaw_paged_i4_read):
        t.call(call)
    assert gqaw.gqaw_launch_count() >= launches + 5
    assert (t.out == 7.0).all() and (t.ko == 7.0).all() and (t.vo == 7.0).all()
    for x, y in zip(t.snapshot(), before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
