"""Keys and values that are not finite, in rows that some new tokens of a paged batch attend and
others do not, on a GB300: every kernel of the attention, and the step with turned queries.  Who
does not attend such a row has the definition's output; who does has one that is not finite.

The rows per kv head choose the kernel: at most 8 the decode kernels, up to 128 one query tile, more
two at once (head sizes 64 and 128)."""
from __future__ import annotations

import pytest
import torch

from paged_driver import Batch
from sliding_window_gqa_02_gb300 import gqaw

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# dtype, head size, page, query heads, kv heads, new tokens
SHAPES = [
    (BF, 64, 16, 8, 2, 2), (BF, 128, 16, 8, 2, 2), (BF, 256, 8, 8, 2, 2),   # decode kernel, 8 rows
    (BF, 64, 64, 2, 2, 4), (BF, 128, 32, 2, 2, 8), (BF, 256, 128, 2, 2, 3),  # ... a head a group
    (F, 32, 16, 8, 2, 2), (F, 64, 16, 2, 2, 8), (F, 128, 16, 4, 2, 2),       # fp32 decode by TMA
    (F, 64, 5, 8, 2, 2), (F, 128, 24, 2, 2, 3), (BF, 64, 24, 8, 2, 2), (BF, 32, 16, 2, 2, 7),  # a warp a tile
    (F, 256, 16, 8, 2, 2), (F, 128, 16, 8, 2, 9), (BF, 16, 16, 8, 2, 40),    # rows on the CUDA cores
    (BF, 64, 16, 8, 2, 20), (BF, 128, 16, 8, 2, 30), (BF, 256, 16, 8, 2, 9), (BF, 256, 16, 8, 2, 70),  # one query tile
    (BF, 64, 16, 8, 2, 90), (BF, 128, 16, 8, 2, 70), (BF, 128, 128, 8, 1, 100),  # two at once
]
IDS = ["%s-%d-%d-%d-%d-%d" % ((str(s[0])[6:],) + s[1:]) for s in SHAPES]


def _place(b, i, j, value, keys=False):
    """A value (or key) row of position j of sequence i, in part."""
    (b.kp if keys else b.vp)[int(b.table[i, j // b.page]), :, j % b.page, 3::5] = value


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_values(shape, window, value):
    dtype, D, page, Nq, Nkv, S = shape
    lens = [(S, 200), (1, 77), (S, S), (S, 300)]
    b = Batch(lens, Nq, Nkv, D, page, dtype, seed=41, window=window)
    for i in (0, 2, 3):
        T = lens[i][1]
        _place(b, i, T - 1, value)          # the last token's own
        _place(b, i, T - S + S // 2, value)  # half of the tokens attend it
        if window and T > S + window:       # only the first token's window reaches it
            _place(b, i, T - S - window + 1, value)
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_keys(shape, window):
    dtype, D, page, Nq, Nkv, S = shape
    lens = [(S, 200), (1, 77), (S, 300)]
    mk = lambda: Batch(lens, Nq, Nkv, D, page, dtype, seed=42, window=window)
    b, c = mk(), mk()
    at = S // 2
    _place(b, 0, 200 - S + at, NAN, keys=True)
    for x in (b, c):
        x.call(gqaw.gqaw_paged_attend)
    rows = torch.arange(int(b.starts[0]) + at, int(b.starts[1]))
    if window:
        rows = rows[rows - rows[0] < window]
    assert torch.isnan(b.out[rows]).all()
    b.out[rows], b.kp = c.out[rows], c.kp
    b.check_output()


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("kw", [dict(), dict(window=64), dict(softcap=15.0, sink=True)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_steps(shape, kw, value):
    """Among the step's own values, with normed and turned queries (in two parts where bf16)."""
    dtype, D, page, Nq, Nkv, S = shape
    lens = [(S, 150), (0, 9), (S, S), (S, 260)]
    b = Batch(lens, Nq, Nkv, D, page, dtype, seed=43, filled=False, norm=True, rotary=D, **kw)
    for i in (0, 2, 3):
        r = int(b.starts[i])
        b.v[r + S - 1, 1::4] = value
        b.v[r + S // 2, 2::7] = value
    b.call(gqaw.gqaw_paged_step)
    b.check_output(turned=True, parts=2 if dtype == BF else 1)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] // s[4] * s[5] >= 8],
                         ids=[i for s, i in zip(SHAPES, IDS) if s[3] // s[4] * s[5] >= 8])
@pytest.mark.parametrize("many", [False, True], ids=["cut", "many"])
def test_cut_units_and_many(shape, many):
    """Long sequences whose units are cut over CTAs, and so many that a CTA takes several."""
    dtype, D, page, Nq, Nkv, S = shape
    lens = [(S, 150 + 3 * (i % 70)) for i in range(180)] if many else [(S, 9000), (1, 40), (S, 7000)]
    b = Batch(lens, Nq, Nkv, D, page, dtype, seed=44)
    for i, (s, t) in enumerate(lens):
        if s > 1 and i % 3 == 0:
            _place(b, i, t - 1, INF)
            _place(b, i, t - s // 2 - 1, NAN)
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()
    first = b.out.clone()
    b.out.fill_(7.0)
    b.call(gqaw.gqaw_paged_attend)
    assert torch.equal(torch.nan_to_num(first), torch.nan_to_num(b.out))
