"""Attention over 4-bit caches with values of any finite size: every output element against 64 bits, with what
its own row, kv head and group of elements allow it, and not with the largest value of the batch."""
from __future__ import annotations

import math

import pytest
import torch

import paged_reference as ref
from i4_driver import Batch
from sliding_window_gqa_02_gb300 import gqaw

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
LONG = 1 << 20  # a length for which the expanded pages of a few sequences would be too large


def check_rows(t, coarse=True, skip=()):
    """``ref.attend``'s bound, which is relative to sum p |v| of the row and element, with 2^-22 for the queries
    (two parts of fp16 and a power of two), and with the ends of the types:
      - a weight below 2^-126 of the row's largest may count as nothing: 2^-125 |v| a key, for a largest one that is
        rounded up to a power of two;
      - ``coarse``: a weight is held in fp16, the row's largest at 2^12 or more: what is rounded to a multiple of
        2^-24 is off by 2^-25, 2^-37 of it.  Without it where the result may hang on such weights: values far apart, whose
        weights are held in fp32;
      - a result is rounded to a multiple of the smallest number, 2^-133 (bf16; fp32 has more), and so may each of
        the T products be where nothing is scaled: (T + 1) 2^-133.
    Keys and values that some row does not attend have no part in its bound."""
    k_all, v_all = t.held()
    sink = t.sink if t.sink is not None else (torch.zeros(t.Nq, device=t.q.device) if t.smooth else None)
    for i, (s, n) in enumerate(t.lens):
        if s == 0 or i in skip:
            continue
        k, v = (ref.gather(x, t.table[i], n, True) for x in (k_all, v_all))
        q = t.q.reshape(-1, t.Nq, t.D).double()[t.rows(i)]
        want, bound = ref.attend(q, k, v, n - s, t.window, t.scale or 1 / math.sqrt(t.D), t.softcap, sink, t.dtype, 2.0 ** -22)
        j = torch.arange(n, device=q.device)
        at = n - s + torch.arange(s, device=q.device)
        seen = (j[None] <= at[:, None]) & ((j[None] > at[:, None] - t.window) if t.window else (j[None] >= 0))
        size = torch.einsum("st,thd->shd", seen.double(), v.abs()).repeat_interleave(t.Nq // t.Nkv, 1)
        bound = bound + (2.0 ** -125 + (2.0 ** -37 if coarse else 0.0)) * size + (n + 1) * 2.0 ** -133
        assert torch.isfinite(want).all()
        got = t.out[t.rows(i)].reshape(s, t.Nq, t.D).double()
        err = (got - want).abs()
        ok = err <= bound  # a NaN is not
        assert ok.all(), "sequence %d: %d elements, first at %s: %s, expected %s within %s" % (
            i, int((~ok).sum()), torch.nonzero(~ok)[:3].tolist(), got[~ok][:3].tolist(), want[~ok][:3].tolist(), bound[~ok][:3].tolist())


def scale_values(t, i, j, exponent, groups=slice(None)):
    """Value scales of position j of sequence i times 2^exponent."""
    pg, r = int(t.table[i, j // t.page]), j % t.page
    if pg < 0:  # left every window
        return
    row = t.vs[pg, r] if t.hir else t.vs[pg, :, r]
    row[:, groups] = (row[:, groups].double() * 2.0 ** exponent).to(BF16)


# ------------------------------------------------------------------------------ values far apart


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,page", [(32, 16), (64, 16), (128, 16), (128, 24), (256, 32)])
@pytest.mark.parametrize("exponent", [12, 22, 40, 100])
def test_a_later_token_with_large_values(dtype, D, page, exponent):
    """The last drafted token's values are far above all others: the tokens before it do not attend it and keep their bits."""
    t = Batch([(4, 90), (1, 40), (2, 300), (6, 33)], 4, 2, D, page, dtype, seed=31)
    t.call(gqaw.gqaw_paged_i4_attend)
    check_rows(t)
    before = t.out.clone()
    for i in (0, 2, 3):
        scale_values(t, i, t.lens[i][1] - 1, exponent)
    t.call(gqaw.gqaw_paged_i4_attend)
    last = torch.zeros(t.out.shape[0], dtype=torch.bool)
    for i in (0, 2, 3):
        last[t.rows(i).stop - 1] = True
    assert torch.equal(t.out[~last], before[~last])
    check_rows(t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_that_have_left_the_window(dtype, D):
    """Only the first new token still attends a key with large values; and none does."""
    for j in (150 - 6 - 20 + 1, 150 - 6 - 20):
        t = Batch([(6, 150)], 4, 2, D, 16, dtype, seed=32, window=20)
        scale_values(t, 0, j, 60)
        t.call(gqaw.gqaw_paged_i4_attend)
        check_rows(t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("lens", [[(8, 60)], [(1, 60), (8, 2000), (1, 900)], [(13, 200)]])
@pytest.mark.parametrize("order", ["up", "down", "any"])
def test_values_of_every_size(dtype, D, lens, order):
    """Scales from 2^-120 to 2^110 in one context, growing, falling (a window lets the large ones go) and mixed, by
    group; logits that move the softmax's reference on the way."""
    t = Batch(lens, 4, 2, D, 16, dtype, seed=33, scale=0.5, window=7 if order == "down" else 0)
    g = torch.Generator().manual_seed(5)
    for i, (s, n) in enumerate(lens):
        for j in range(n):
            for group in range(D // 32):
                x = j / n * 230
                e = {"up": x - 120, "down": 110 - x, "any": float(torch.randint(-118, 108, (1,), generator=g))}[order]
                scale_values(t, i, j, round(e) - (7 * group if order == "up" else 0), group)
    t.call(gqaw.gqaw_paged_i4_attend)
    check_rows(t, coarse=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [30, 60, 90])
def test_large_values_under_small_weights(dtype, power):
    """A key whose weight is 2^-power of the others' and whose values are 2^power of theirs counts like them."""
    for D in (64, 128):
        t = Batch([(1, 50), (3, 700)], 4, 2, D, 16, dtype, seed=34, scale=1.0)
        t.q.fill_(1.0)
        t.ks.copy_(torch.where(t.ks.isnan(), t.ks, t.ks * 2.0 ** -8))
        for i, j in ((0, 20), (1, 333), (1, 40)):
            pg, r = int(t.table[i, j // 16]), j % 16
            t.kc[pg, :, r] = 0x77  # every element -1 times the scale
            t.ks[pg, :, r] = power * math.log(2) / D
            scale_values(t, i, j, power)
        t.call(gqaw.gqaw_paged_i4_attend)
        check_rows(t, coarse=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_groups_heads_and_pages_far_apart(dtype):
    """Groups, heads and pages of very different sizes, each held to its own."""
    t = Batch([(1, 300), (6, 140)], 4, 2, 128, 16, dtype, seed=35)
    f = 10.0 ** torch.randint(-9, 10, (t.vs.shape[0], 2, 1, 1))
    e = torch.tensor([1e-12, 1.0, 1e12, 1e-3]).reshape(1, 1, 1, 4)
    t.vs.copy_((t.vs.double().cpu() * f * e).to(BF16))
    t.call(gqaw.gqaw_paged_i4_attend)
    check_rows(t, coarse=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales_that_are_not_finite_among_values_of_every_size(dtype):
    """Scales that are not finite still reach their own group of the tokens that attend them, and nothing else."""
    t = Batch([(4, 80)], 4, 2, 128, 16, dtype, seed=36, window=30)
    for j in range(80):
        scale_values(t, 0, j, (j * 37) % 200 - 100)
    t.call(gqaw.gqaw_paged_i4_attend)
    check_rows(t, coarse=False)
    before = t.out.clone().reshape(4, 4, 4, 32)
    for j, bad in ((78, float("inf")), (48, float("nan"))):  # the last two tokens attend 78, the first two 48
        t.vs[int(t.table[0, j // 16]), 1, j % 16, 2] = bad
    t.call(gqaw.gqaw_paged_i4_attend)
    after = t.out.reshape(4, 4, 4, 32)
    same = torch.ones(4, 4, 4, dtype=torch.bool)
    same[:, 2:, 2] = False
    assert torch.equal(after[same], before[same])
    assert not after[~same].isfinite().any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_groups_that_begin_with_zeros(dtype, D):
    """Values of zero in a warp's first tiles, in one group or in all; small ones behind them."""
    t = Batch([(1, 2000), (5, 700)], 4, 2, D, 16, dtype, seed=42)
    for i, n in ((0, 1500), (1, 690)):
        for j in range(n):
            pg = int(t.table[i, j // 16])
            t.vs[pg, 0, j % 16, 0] = 0.0
            t.vs[pg, 1, j % 16] = -0.0
    t.call(gqaw.gqaw_paged_i4_attend)
    check_rows(t)


def test_a_row_attends_the_same_whatever_others_attend():
    """Drafts of one to eight tokens at the same place: a token's bits do not hang on how many follow it, nor on how large
    their values are."""
    D, n = 128, 200
    t = Batch([(1, n)], 4, 2, D, 16, BF16, seed=43, extra_rows=7, max_len=n + 8)
    full = Batch([(8, n + 7)], 4, 2, D, 16, BF16, seed=44)
    full.q[0] = t.q[0]
    for a, b in ((t.kc, full.kc), (t.vc, full.vc), (t.ks, full.ks), (t.vs, full.vs)):
        for j in range(n):
            b[int(full.table[0, j // 16]), :, j % 16] = a[int(t.table[0, j // 16]), :, j % 16]
    t.call(gqaw.gqaw_paged_i4_attend)
    for j in range(n, n + 7):
        scale_values(full, 0, j, 3 * (j - n) * 6)
    full.call(gqaw.gqaw_paged_i4_attend)
    check_rows(full)
    diff = (t.out[0].double() - full.out[0].double()).abs()
    assert (diff <= 2.0 ** -8 * t.out[0].double().abs() + 2.0 ** -9 * t.out[0].double().abs().max()).all()


# ------------------------------------------------------------------------------ values near the type's end


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kw", [dict(), dict(sink=True), dict(softcap=3.0), dict(window=100)])
def test_values_near_the_end_of_the_type(dtype, kw):
    """Elements up to 2e38 whose averages are finite, by rows: one CTA's units, cut ones, few and many keys."""
    for D, lens in ((64, [(1, 300), (2, 9000), (8, 8)]), (128, [(1, 5000), (1, 1), (6, 40)]), (256, [(2, 700)]), (32, [(3, 90)])):
        t = Batch(lens, 4, 2, D, 16, dtype, seed=37, **kw)
        t.vs.copy_((t.vs.double() * 2.0 ** 125.5).to(BF16))
        assert t.held()[1].nan_to_num(0.0).abs().max() < 3.3e38
        t.call(gqaw.gqaw_paged_i4_attend)
        check_rows(t)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_key_near_the_end_of_the_type(dtype):
    """One value of 2^125 among small ones, under an ordinary weight."""
    t = Batch([(1, 3000), (3, 70)], 4, 2, 128, 16, dtype, seed=38)
    scale_values(t, 0, 1234, 125)
    scale_values(t, 1, 5, 125)
    t.call(gqaw.gqaw_paged_i4_attend)
    check_rows(t)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_long_context_of_large_values(dtype):
    """The same sign everywhere and weights alike: sums over 40,000 keys of what is near the type's end."""
    t = Batch([(1, 40000)], 2, 1, 64, 64, dtype, seed=45)
    t.q.fill_(0.0)
    t.vc.fill_(0xFF)
    for power in (62, 70, 100, 125):
        t.vs.copy_(torch.where(t.vs.isnan(), t.vs, torch.full_like(t.vs, 2.0 ** power)))
        t.call(gqaw.gqaw_paged_i4_attend)
        check_rows(t)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_len", [0, LONG])
def test_chunks_with_one_large_value(D, max_len):
    """Prompt chunks, on expanded keys and on codes: a key with elements up to 1.4e38 (a scale that times 24 leaves the
    type), which some tokens do not attend and the others attend with a weight of 2^-30."""
    t = Batch([(200, 300), (100, 100), (70, 70), (90, 91)], 8, 2, D, 16, BF16, seed=39, max_len=max_len, scale=1.0)
    t.q.fill_(1.0)
    t.ks.copy_(torch.where(t.ks.isnan(), t.ks, t.ks * 2.0 ** -8))
    for i, j in ((0, 180), (1, 60)):
        pg, r = int(t.table[i, j // 16]), j % 16
        t.kc[pg, :, r] = 0x77
        t.ks[pg, :, r] = 30 * math.log(2) / D
        t.vs[pg, :, r] = 1.1 * 2.0 ** 124
        t.vs.view(torch.int16)[pg, :, r] &= ~7  # five significant bits, as the append writes them
    t.call(gqaw.gqaw_paged_i4_attend)
    check_rows(t, coarse=False)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_len", [0, LONG])
def test_chunks_with_large_keys(D, max_len):
    """Keys near the end of the type under queries near the other."""
    t = Batch([(200, 300), (100, 100), (70, 70), (90, 91)], 8, 2, D, 16, BF16, seed=40, max_len=max_len, scale=1.0)
    t.ks.copy_((t.ks.double() * 2.0 ** 125.5).to(BF16))
    t.ks.view(torch.int16)[:] &= ~7
    t.ks.copy_(t.ks.nan_to_num(0.25))
    t.q.copy_((t.q.double() * 2.0 ** -124 / D).to(BF16))
    t.call(gqaw.gqaw_paged_i4_attend)
    check_rows(t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_large_queries_beside_small_ones_over_large_keys(dtype, D):
    """A very large row, whose own logits may leave fp32, and very small ones over very large keys: the small ones have
    ordinary logits and keep their bits."""
    t = Batch([(3, 90), (1, 700)], 4, 2, D, 16, dtype, seed=46, scale=1.0)
    t.ks.copy_((t.ks.double() * 2.0 ** 110).to(BF16))
    t.q.copy_((t.q.double() * 2.0 ** -112).to(dtype))
    t.call(gqaw.gqaw_paged_i4_attend)
    check_rows(t)
    before = t.out.clone().reshape(-1, 4, D)
    for value in (2.0 ** 20, 2.0 ** 70, 1e30, 3e38, float("inf")):
        t.q[1, D + 5] = value  # token 1, head 1
        t.call(gqaw.gqaw_paged_i4_attend)
        after = t.out.reshape(-1, 4, D)
        same = torch.ones(4, 4, dtype=torch.bool)
        same[1, 1] = False
        assert torch.equal(after[same], before[same])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("f", [1e-30, 1e-10, 1e5, 1e20, 1e25, 1e30, 1e36])
def test_rows_of_queries_of_every_size(dtype, f):
    """Queries of size f with keys to match, among rows a thousand times smaller."""
    for D, S in ((64, 3), (128, 8), (256, 1)):
        t = Batch([(S, 300), (1, 40)], 4, 2, D, 16, dtype, seed=47, scale=1.0)
        t.q.copy_((t.q.double() * f).to(dtype))
        t.q.view(-1, 4, D)[:, 1::2] /= 1000
        t.ks.copy_((t.ks.double() / f / 8).to(BF16))
        t.call(gqaw.gqaw_paged_i4_attend)
        check_rows(t)
