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


# rows per sequence as built, query_start as given, and the sequences that are not malformed
DESCENDING = {
    # the last sequence starts in the first's rows, and has more than any may
    "past the first": ([(50, 50), (10, 20), (0, 0), (48, 200)], [0, 50, 60, 3, 108], (0, 1)),
    "short": ([(4, 31), (4, 11), (0, 6), (1, 21)], [0, 4, 8, 1, 9], (0, 1)),
    "one row left": ([(2, 30), (3, 40), (1, 90)], [0, 6, 5, 6], (2,)),
    "below the first": ([(3, 40), (0, 7), (1, 33), (0, 0)], [10, 13, 3, 4, 4], (0, 2, 3)),
    "many": ([(2, 20 + i) for i in range(90)], [2 * i if i != 40 else 5 for i in range(91)], tuple(i for i in range(90) if i not in (39, 40))),
}


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("case", DESCENDING)
@pytest.mark.parametrize("call", ["gqaw_paged_append", "gqaw_paged_step"])
def test_starts_that_descend(call, case, dtype):
    """Every row goes to its own sequence: no other page row changes, wherever the starts point."""
    lens, starts, right = DESCENDING[case]
    b = Batch(lens, 4, 2, 64, 16, dtype, seed=32, filled=False, lead_rows=10 if starts[0] else 0, norm=True, rotary=64)
    b.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    for i in right:  # row by row the positions of the sequences that are right
        s, t = lens[i]
        b.pos[starts[i]:starts[i] + s] = torch.arange(t - s, t)
    k0, v0 = b.kp.clone(), b.vp.clone()
    b.call(getattr(gqaw, call), flags=gqaw.GQAW_DEV_BAD_SEQLEN)
    b.lens = [x if i in right else (0, x[1]) for i, x in enumerate(lens)]
    b.check_pages(k0, v0)
    if call == "gqaw_paged_step":
        b.check_output(turned=True, parts=2 if dtype == BF else 1)
        b.check_untouched()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("call", ["gqaw_paged_append", "gqaw_paged_step"])
def test_shared_rows_touch_only_their_sequences(call, dtype):
    """Sequences that claim the same rows and are well formed otherwise: what they get is not
    specified, but it stays in their own new positions, and a sequence beside them is right."""
    lens = [(50, 64), (10, 20), (0, 0), (57, 200), (5, 70)]
    b = Batch(lens, 4, 2, 64, 16, dtype, seed=33, filled=False)
    b.starts = torch.tensor([0, 50, 60, 3, 60, 65], dtype=torch.int32, device="cuda")
    b.q, b.k, b.v, b.out = (x[:65].contiguous() for x in (b.q, b.k, b.v, b.out))
    b.pos = b.pos[:65]
    b.pos[60:] = torch.arange(65, 70)
    k0, v0 = b.kp.clone(), b.vp.clone()
    b.call(getattr(gqaw, call), flags=gqaw.GQAW_DEV_BAD_SEQLEN)
    for i in (0, 1, 3):
        s, t = lens[i]
        j = torch.arange(t - s, t, device="cuda")
        pg, at = b.table[i].long()[j // 16], j % 16
        for now, before in ((b.kp, k0), (b.vp, v0)):
            now[pg, :, at] = before[pg, :, at]
    b.lens = [(s if i == 4 else 0, t) for i, (s, t) in enumerate(lens)]
    b.check_pages(k0, v0)
    if call == "gqaw_paged_step":
        b.check_output()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D,S", [(64, 1), (64, 40), (256, 1), (32, 3)])
def test_a_cache_without_pages(D, S, dtype):
    """No page exists: every table entry is out of range, and the tokens' outputs are unspecified."""
    b = Batch([(S, 40), (0, 5), (1, 9)], 4, 2, D, 16, dtype, seed=34, norm=True, rotary=D, extra_rows=2)
    b.kp, b.vp = b.kp[:0], b.vp[:0]
    assert b.args().num_pages == 0
    for call in (gqaw.gqaw_paged_append, gqaw.gqaw_paged_attend, gqaw.gqaw_paged_step):
        b.call(call, flags=gqaw.GQAW_DEV_BAD_PAGE)
    assert (b.out[S + 1:] == 7.0).all()
    c = Batch([(S, 40), (1, 9)], 4, 2, D, 16, dtype, seed=35)
    c.call(gqaw.gqaw_paged_attend)
    c.check_output()
