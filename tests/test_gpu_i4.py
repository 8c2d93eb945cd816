"""The operators on 4-bit paged caches on a GPU: codes bit for bit, outputs against 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import i4_reference as i4
from i4_driver import Batch
from sliding_window_gqa_02_gb300 import gqaw

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

RAGGED = [(1, 1), (3, 17), (0, 40), (0, 0), (33, 33), (5, 70), (1, 64), (16, 49)]


# ------------------------------------------------------------------------------ append and read


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,Nq,Nkv,page", [(32, 3, 3, 7), (64, 8, 2, 16), (128, 6, 1, 1), (128, 16, 8, 32), (256, 5, 5, 24)])
def test_append_and_read(dtype, D, Nq, Nkv, page):
    t = Batch(RAGGED, Nq, Nkv, D, page, dtype, seed=D + page, extra_rows=3, lead_rows=2, filled=False)
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_append)
    t.check_pages(before)
    t.call(gqaw.gqaw_paged_i4_read)
    t.check_read()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,rotary,inter", [(128, 128, False), (128, 64, True), (64, 24, False), (64, 22, True), (256, 256, False),
                                           (32, 6, False), (32, 32, True), (128, 100, False), (256, 4, False)])
def test_append_norm_turn(dtype, D, rotary, inter):
    t = Batch(RAGGED, 4, 2, D, 16, dtype, seed=rotary, norm=True, rotary=rotary, interleaved=inter, filled=False,
              position_ids=D == 64, fused=D == 128, lead_rows=1)
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_append)
    t.check_pages(before)


@pytest.mark.parametrize("norm,rotary", [(True, 0), (False, 64), (False, 16)])
def test_append_norm_or_turn(norm, rotary):
    t = Batch(RAGGED, 4, 2, 64, 16, BF16, seed=5, norm=norm, rotary=rotary, filled=False)
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_append)
    t.check_pages(before)


def test_append_many_rows():
    """More rows than the kernel with two groups a warp takes, in fp32 and bf16, heads not a multiple of a warp's."""
    for dtype, D, Nkv in ((BF16, 128, 5), (F32, 64, 3)):
        t = Batch([(700, 700), (1, 900), (513, 1000)], Nkv, Nkv, D, 64, dtype, seed=3, norm=True, rotary=D, filled=False)
        before = t.snapshot()
        t.call(gqaw.gqaw_paged_i4_append)
        t.check_pages(before)
        t.call(gqaw.gqaw_paged_i4_read)
        t.check_read()


def test_append_values_at_the_edges():
    """Zeros, the smallest and largest numbers, infinities and NaN, ties between codes, one large element."""
    t = Batch([(16, 16)], 1, 1, 128, 16, F32, filled=False)
    v = torch.randn(16, 128)
    v[0] = 0.0
    v[1] = 1e-45
    v[2, :40] = 3.4e38
    v[3, 5] = float("inf")
    v[4, 100] = float("nan")
    v[5, 64] = float("-inf")
    v[6] = torch.arange(128) % 15 - 7.0          # exact codes, scale 1
    v[7] = (torch.arange(128) % 14 - 7.0) + 0.5  # ties
    v[7, ::32] = 7.0
    v[8] = 1e-40
    v[9, 0::32] = 1e30
    v[10] = -0.0
    v[11] *= 1e-38
    v[12] *= 2.0 ** -126
    v[13] = 7.0 * 1.0625 * 2.0 ** -140
    t.v.copy_(v)
    t.k.copy_(v.flip(0))
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_append)
    t.check_pages(before)
    t.call(gqaw.gqaw_paged_i4_read)
    t.check_read()
    back = t.vo.cpu()
    assert torch.equal(back[6], v[6]) and (back[0] == 0).all() and back[3, :32].isnan().all() and (back[3, 32:64] != 7).any()


def test_append_turn_rounds_each_operation():
    """Elements that lie on the border of two codes when every product and sum of the turn is rounded, and
    below it when a product is contracted with the sum: a c - b with b = fl(a c) - 3.5 scale."""
    rng = np.random.default_rng(1)
    t = Batch([(64, 64)], 1, 1, 32, 16, F32, rotary=2, position_ids=True, filled=False)
    rows = t.cos.shape[0]
    a, c = np.zeros(rows, np.float32), np.zeros(rows, np.float32)
    i = 0
    while i < rows:
        x, y = (rng.random(2) * 0.5 + 1.0).astype(np.float32)
        p = x * y
        if np.float64(x) * np.float64(y) < np.float64(p):  # the rounded product lies above
            a[i], c[i] = x, y
            i += 1
    s = np.float32(1.25)
    b = a * c - np.float32(3.5) * s
    assert (a * c - b == np.float32(3.5) * s).all()
    ids = np.arange(64) % rows
    x = np.zeros((64, 32), np.float32)
    x[:, 0], x[:, 1], x[:, 2] = a[ids], b[ids], 7 * s
    t.cos.copy_(torch.from_numpy(c)[:, None])
    t.sin.fill_(1.0)
    t.ids = torch.from_numpy(ids).to(t.k.device)
    t.k.copy_(torch.from_numpy(x))
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_append)
    t.check_pages(before)
    t.call(gqaw.gqaw_paged_i4_read)
    assert (t.ko[:, 0] == 4 * float(s)).all()


def test_append_norm_far_rows():
    """Rows whose squares leave fp32 on either side are normed in 64 bits; so is a row of zeros."""
    t = Batch([(8, 8)], 1, 1, 64, 16, F32, norm=True, filled=False)
    x = torch.randn(8, 64)
    for i, f in enumerate((1.0, 1e25, 1e-25, 3e38 / 6, 1e-38, 0.0, 1e-3, 1e3)):
        t.k[i] = (x[i] * f).to(t.k.device)
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_append)
    t.check_pages(before)


def test_error_of_a_row():
    """What the cache holds is within half a scale of the row, and a scale at most 17 / 16 of its group's
    largest element over 7."""
    t = Batch([(64, 64)], 4, 4, 128, 16, BF16, filled=False)
    t.call(gqaw.gqaw_paged_i4_append)
    t.call(gqaw.gqaw_paged_i4_read)
    for x, y in ((t.k, t.ko), (t.v, t.vo)):
        x, y = (a.double().reshape(64, 4, 4, 32) for a in (x, y))
        top = x.abs().amax(-1)
        # the quotient, the division and the stored value are exact to 2^-23; five bits are a step of 1 / 16
        limit = top / 7 * 17 / 16 * (1 + 2.0 ** -22) / 2
        assert ((x - y).abs() <= limit[..., None] * (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("kw", [dict(heads_inside_rows=True), dict(woven=True), dict(heads_inside_rows=True, woven=True)])
def test_layouts(kw):
    for D, dtype in ((128, BF16), (32, F32)):
        t = Batch(RAGGED, 4, 2, D, 16, dtype, seed=9, norm=True, rotary=32, **kw)
        before = t.snapshot()
        t.call(gqaw.gqaw_paged_i4_step)
        t.check_pages(before)
        t.check_output(turned=True)
        t.call(gqaw.gqaw_paged_i4_read)
        t.check_read()


def test_read_one_tensor_only():
    t = Batch(RAGGED, 4, 2, 64, 16, BF16)
    t.call(gqaw.gqaw_paged_i4_read, value_out=None)
    t.check_read(vals=False)
    t = Batch(RAGGED, 4, 2, 64, 16, BF16)
    t.call(gqaw.gqaw_paged_i4_read, key_out=None)
    t.check_read(keys=False)


def test_read_into_one_tensor():
    t = Batch(RAGGED, 4, 2, 64, 16, BF16)
    both = torch.full((t.ko.shape[0], 2, 128), 7.0, dtype=BF16, device=t.ko.device)
    t.ko, t.vo = both[:, 0], both[:, 1]
    t.call(gqaw.gqaw_paged_i4_read)
    t.check_read()


# ------------------------------------------------------------------------------ attention


SHAPES = [(32, 4, 2, 16), (64, 8, 1, 16), (128, 8, 2, 16), (256, 4, 4, 32), (128, 7, 1, 24), (64, 5, 5, 3), (128, 8, 2, 128), (64, 12, 3, 1)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,Nq,Nkv,page", SHAPES)
@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 131), (1, 700), (1, 16), (1, 257)], [(2, 33), (4, 100), (0, 9), (1, 513)]])
def test_attend_few_rows(dtype, D, Nq, Nkv, page, lens):
    t = Batch(lens, Nq, Nkv, D, page, dtype, seed=D, extra_rows=2, lead_rows=1)
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()
    assert (t.out[t.untouched()] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,Nq,Nkv,page", SHAPES)
@pytest.mark.parametrize("opt", [dict(), dict(window=50, sink=True), dict(softcap=5.0, scale=0.3, window=9)])
def test_attend_chunks(dtype, D, Nq, Nkv, page, opt):
    t = Batch([(33, 33), (1, 300), (70, 200), (0, 5), (129, 401), (8, 8)], Nq, Nkv, D, page, dtype, seed=page, **opt)
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()


LONG = 1 << 20  # a length for which the expanded pages of a few sequences would be too large


@pytest.mark.parametrize("D,Nq,Nkv,page", SHAPES)
@pytest.mark.parametrize("opt", [dict(), dict(window=LONG - 1, sink=True), dict(softcap=5.0, scale=0.3)])
def test_attend_chunks_of_batches_that_may_be_long(D, Nq, Nkv, page, opt):
    """The prompt kernel that takes codes, whose choice goes by the longest length that the call allows."""
    t = Batch([(33, 33), (1, 300), (70, 200), (0, 5), (129, 401), (8, 8)], Nq, Nkv, D, page, BF16, seed=page, max_len=LONG, **opt)
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()


@pytest.mark.parametrize("max_len", [0, LONG])
@pytest.mark.parametrize("kw", [dict(odd_scales=True), dict(norm=True, rotary=64), dict(window=70, sink=True), dict(heads_inside_rows=True)])
def test_chunks_either_way(max_len, kw):
    """Chunks of several query tiles, with their keys expanded beforehand and as codes."""
    for D, Nq, Nkv, page in ((128, 8, 2, 16), (64, 16, 1, 24)):
        t = Batch([(200, 300), (1, 90), (300, 300), (2, 2)], Nq, Nkv, D, page, BF16, seed=3, max_len=max_len, lead_rows=1, extra_rows=2, **kw)
        t.call(gqaw.gqaw_paged_i4_step)
        t.check_output(turned=True)
        assert (t.out[t.untouched()] == 7.0).all()


@pytest.mark.parametrize("max_len", [0, 8192, LONG])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks_by_the_work_that_a_call_may_be(D, max_len):
    """The same chunks by rows, with expanded keys (head size 256) and as codes: a call chooses by the longest
    sequences that it allows."""
    t = Batch([(32, 300), (1, 90), (20, 1000), (2, 2)], 8, 2, D, 16, BF16, seed=3, max_len=max_len, lead_rows=1, extra_rows=2)
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()
    assert (t.out[t.untouched()] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("opt", [dict(window=1), dict(window=100, softcap=30.0), dict(sink=True), dict(smooth=True, softcap=2.0),
                                 dict(scale=2.0), dict(odd_scales=True), dict(odd_scales=True, window=33)])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 65), (1, 1)], [(8, 300), (3, 130), (8, 8)], [(40, 300), (100, 100)]])
def test_attend_options(dtype, opt, lens):
    t = Batch(lens, 8, 2, 128, 16, dtype, seed=1, **opt)
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 16, 31, 33, 64, 130])
def test_attend_groups(group):
    for dtype, S in ((BF16, 1), (BF16, 5), (F32, 2)):
        t = Batch([(S, 150), (1, 77)], 2 * group, 2, 64, 16, dtype, seed=group)
        t.call(gqaw.gqaw_paged_i4_attend)
        t.check_output()


def test_attend_long_contexts_split_between_ctas():
    for dtype, Nq, Nkv, D in ((BF16, 8, 2, 128), (F32, 8, 1, 64), (BF16, 4, 1, 256)):
        t = Batch([(1, 9000), (1, 4097), (2, 20000), (1, 31)], Nq, Nkv, D, 64, dtype, seed=2)
        t.call(gqaw.gqaw_paged_i4_attend)
        t.check_output()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_scales_far_apart(dtype):
    """Scales of very different sizes, by group, by key and by head: no group loses bits to another's."""
    t = Batch([(1, 300), (6, 140)], 4, 2, 128, 16, dtype, seed=4)
    f = 10.0 ** torch.randint(-9, 10, (t.vs.shape[0], 2, 1, 1))
    t.vs.copy_((t.vs.float().cpu() * f).to(BF16))
    e = torch.tensor([1e-12, 1.0, 1e12, 1e-3]).reshape(1, 1, 1, 4)
    t.vs.copy_((t.vs.float().cpu() * e).to(BF16))
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_queries_of_any_size(dtype):
    """Rows of queries from 1e-20 to 1e20, and one element far above the others, with keys to match."""
    for f in (1e-20, 1e20, 3e37):
        t = Batch([(1, 200), (3, 90)], 4, 2, 64, 16, dtype, seed=6, scale=1.0)
        t.q.copy_((t.q.float() * f).to(dtype))
        t.ks.copy_((t.ks.float() / f / 8).to(BF16))
        t.call(gqaw.gqaw_paged_i4_attend)
        t.check_output()
    t = Batch([(1, 200)], 4, 2, 64, 16, dtype, seed=6)
    t.q[:, ::64] *= 1000
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3e37, -1e30])
def test_attend_one_query_row_does_not_reach_the_others(dtype, value):
    """A head of one token that is not finite or very large, beside large keys: other rows keep their bits."""
    for D in (64, 128):
        t = Batch([(3, 90), (1, 40)], 4, 2, D, 16, dtype, seed=12, scale=2.0 ** -20)
        t.ks.copy_((t.ks.float() * 2.0 ** 20).to(BF16))
        t.call(gqaw.gqaw_paged_i4_attend)
        t.check_output()
        before = t.out.clone().reshape(-1, 4, D)
        t.q[1, D + 5] = value  # token 1, head 1
        t.call(gqaw.gqaw_paged_i4_attend)
        after = t.out.reshape(-1, 4, D)
        same = torch.ones(4, 4, dtype=torch.bool)
        same[1, 1] = False
        assert torch.equal(after[same], before[same])
        if value != value or abs(value) == float("inf"):
            assert after[1, 1].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S,max_len", [(1, 0), (6, 0), (40, 0), (70, 0), (70, LONG)])
def test_attend_scales_that_are_not_finite(dtype, S, max_len):
    """A value scale that is NaN or infinite reaches the 32 elements of its group in the outputs of tokens that
    attend it, and nothing else."""
    t = Batch([(S, 180), (S, 75)], 4 if S < 70 else 8, 2, 128, 16, dtype, seed=8, window=60, max_len=max_len)
    half = t.Nq // 2
    pos = {0: 180 - S // 2 - 1, 1: 75 - S}
    for i, j in pos.items():
        pg = int(t.table[i, j // 16])
        t.vs[pg, 1, j % 16, 2] = float("nan") if i == 0 else float("inf")
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()
    for i, j in pos.items():
        rows = t.out[t.rows(i)].reshape(S, t.Nq, 4, 32)
        first = t.lens[i][1] - S
        for s in range(S):
            sees = first + s >= j and j > first + s - 60
            assert rows[s, half:, 2].isfinite().any() != sees
            assert rows[s, :half].isfinite().all() and rows[s, half:, :2].isfinite().all() and rows[s, half:, 3].isfinite().all()
            if not sees:
                assert rows[s].isfinite().all()


# ------------------------------------------------------------------------------ the step, and a run of all


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [[(1, 40), (1, 1), (1, 300)], [(4, 40), (8, 8), (1, 90)], [(64, 64), (33, 200), (1, 70), (0, 3)]])
@pytest.mark.parametrize("norm,rotary,inter", [(True, 128, False), (False, 64, True), (True, 0, False), (False, 0, False)])
def test_step(dtype, lens, norm, rotary, inter):
    t = Batch(lens, 8, 2, 128, 16, dtype, seed=11, norm=norm, rotary=rotary, interleaved=inter, lead_rows=1, extra_rows=2)
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_step)
    t.check_pages(before)
    t.check_output(turned=True)


def test_a_run_of_prompt_decode_and_read():
    """A prompt in two chunks, decode steps, drafts, the whole sequence read back and attended as bf16
    pages: the same keys and values, so the same outputs."""
    D, Nq, Nkv, page, T = 128, 8, 2, 16, 120
    dev = torch.device("cuda:0")
    sizes = [64, 40, 1, 1, 4, 1, 8, 1]
    t = Batch([(T, T)], Nq, Nkv, D, page, BF16, seed=12, norm=True, rotary=D, filled=False)
    q, k, v = t.q.clone(), t.k.clone(), t.v.clone()
    t.args()  # a workspace for the whole sequence, which serves every smaller call
    at = 0
    outs = []
    for s in sizes:
        t.lens = [(s, at + s)]
        t.q, t.k, t.v = q[at:at + s], k[at:at + s], v[at:at + s]
        t.out = torch.full((s, Nq * D), 7.0, dtype=BF16, device=dev)
        t.ko, t.vo = (torch.full((s, Nkv * D), 7.0, dtype=BF16, device=dev) for _ in "kv")
        t.starts = torch.tensor([0, s], dtype=torch.int32, device=dev)
        t.seqlens = torch.tensor([at + s - 1], dtype=torch.int32, device=dev)
        t.max_new, t.pos = s, torch.arange(at, at + s)
        t.call(gqaw.gqaw_paged_i4_step)
        t.check_output(turned=True)
        outs.append(t.out)
        at += s
    assert at == sum(sizes) <= T
    n = at
    t.lens, t.q, t.k, t.v, t.out = [(n, n)], q[:n], k[:n], v[:n], torch.full((n, Nq * D), 7.0, dtype=BF16, device=dev)
    t.ko, t.vo = (torch.full((n, Nkv * D), 7.0, dtype=BF16, device=dev) for _ in "kv")
    t.starts, t.max_new, t.pos = torch.tensor([0, n], dtype=torch.int32, device=dev), n, torch.arange(n)
    t.call(gqaw.gqaw_paged_i4_read)
    t.check_read()
    # the rows read back, in bf16 pages, under the same queries
    pages = (n + page - 1) // page
    kp, vp = (torch.zeros(pages * page, Nkv, D, dtype=BF16, device=dev) for _ in "kv")
    kp[:n], vp[:n] = t.ko.view(n, Nkv, D), t.vo.view(n, Nkv, D)
    kp, vp = (x.view(pages, page, Nkv, D).contiguous() for x in (kp, vp))
    table = torch.arange(pages, dtype=torch.int32, device=dev)[None].contiguous()
    qn = torch.empty_like(t.q)
    stream = torch.cuda.current_stream().cuda_stream
    gqaw.check(gqaw.gqaw_qk_norm_rotary(gqaw.make_qk_args(t.q, None, qn, None, Nq, 0, D, query_weight=t.qw, norm_eps=1e-5,
                                                          cos_cache=t.cos, sin_cache=t.sin, position_ids=t.pos.to(dev),
                                                          workspace=t.ws), stream))
    out = torch.empty_like(t.out)
    mk = lambda ws: gqaw.make_paged_args(qn, None, None, kp, vp, table, t.starts, t.seqlens, n, n, Nq, Nkv, out,
                                         workspace=ws, heads_inside_rows=True)
    ws = gqaw.new_paged_workspace(mk(None), dev, stream)
    gqaw.check(gqaw.gqaw_paged_attend(mk(ws), stream))
    torch.cuda.synchronize()
    # both within a few roundings to bf16 of the same numbers: queries, weights, outputs
    diff = (torch.cat(outs).double() - out.double()).norm() / out.double().norm()
    assert diff < 4 * 2.0 ** -8


@pytest.mark.parametrize("dtype,S,max_len", [(BF16, 3, 0), (BF16, 70, 0), (BF16, 60, LONG), (F32, 20, 0)])
def test_offsets_past_32_bits(dtype, S, max_len):
    """Pages a gigabyte apart, codes and scales: every path finds its rows."""
    t = Batch([(S, 90), (1, 40)], 8, 2, 64, 32, dtype, seed=21, max_len=max_len, norm=True, rotary=64)
    far = []
    for x, stride in ((t.kc, 1 << 30), (t.vc, 1 << 30), (t.ks, (1 << 30) + 64), (t.vs, (1 << 30) + 64)):
        n = x.shape[0]
        buf = torch.empty((n - 1) * stride + x[0].numel(), dtype=x.dtype, device=x.device)
        y = buf.as_strided(x.shape, (stride, *x.stride()[1:]))
        y.copy_(x)
        far.append(y)
    t.kc, t.vc, t.ks, t.vs = far
    assert far[0].shape[0] > 5
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_step)
    t.check_pages(before)
    t.check_output(turned=True)
    t.call(gqaw.gqaw_paged_i4_read)
    t.check_read()


# ------------------------------------------------------------------------------ malformed, graphs, streams


def test_malformed_sequences_and_bad_pages():
    lens = [(2, 40), (3, 50), (1, 20), (2, 33)]
    t = Batch(lens, 4, 2, 64, 16, BF16, seed=13)
    t.seqlens[1] = 0  # shorter than its new tokens
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_append, flags=gqaw.GQAW_DEV_BAD_SEQLEN)
    t.call(gqaw.gqaw_paged_i4_attend, flags=gqaw.GQAW_DEV_BAD_SEQLEN)
    t.check_output(skip=(1,))
    assert (t.out[t.rows(1)] == 7.0).all()
    t.call(gqaw.gqaw_paged_i4_read, flags=gqaw.GQAW_DEV_BAD_SEQLEN)
    assert (t.ko[t.rows(1)] == 7.0).all()
    t = Batch(lens, 4, 2, 64, 16, BF16, seed=13)
    t.table[3, 2] = 1 << 20  # the page of the last sequence's last token
    t.table[0, 2] = -1
    before = t.snapshot()
    t.call(gqaw.gqaw_paged_i4_append, flags=gqaw.GQAW_DEV_BAD_PAGE)
    t.table[3, 2] = -1
    t.check_pages(before)
    t.call(gqaw.gqaw_paged_i4_attend, flags=gqaw.GQAW_DEV_BAD_PAGE)
    t.check_output(skip=(0, 3))
    t.call(gqaw.gqaw_paged_i4_read, flags=gqaw.GQAW_DEV_BAD_PAGE)
    t.check_read()


@pytest.mark.parametrize("D,max_len", [(128, 0), (64, LONG), (256, 0)])
def test_malformed_chunks_and_bad_pages(D, max_len):
    """The same where prompt kernels run, on expanded keys and on codes."""
    lens = [(100, 300), (120, 200), (1, 20), (90, 333)]
    t = Batch(lens, 8, 2, D, 16, BF16, seed=14, max_len=max_len, lead_rows=1, extra_rows=3)
    t.seqlens[1] = 5  # shorter than its new tokens
    t.call(gqaw.gqaw_paged_i4_attend, flags=gqaw.GQAW_DEV_BAD_SEQLEN)
    t.check_output(skip=(1,))
    assert (t.out[t.rows(1)] == 7.0).all() and (t.out[t.untouched()] == 7.0).all()
    t = Batch(lens, 8, 2, D, 16, BF16, seed=14, max_len=max_len)
    t.seqlens[3] = t.max_len  # longer than the call allows
    t.table[0, 2], t.table[0, 3] = 1 << 20, -1
    t.call(gqaw.gqaw_paged_i4_attend, flags=gqaw.GQAW_DEV_BAD_SEQLEN | gqaw.GQAW_DEV_BAD_PAGE)
    t.check_output(skip=(0, 3))
    assert (t.out[t.rows(3)] == 7.0).all()


@pytest.mark.parametrize("max_len", [0, LONG])
def test_chunks_of_more_sequences_than_one_launch_takes(max_len):
    lens = [(70, 70 + i) if i % 60 == 7 else (i % 3, 20 + i) for i in range(300)]
    t = Batch(lens, 4, 1, 64, 32, BF16, seed=19, max_len=max_len)
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()


def test_graphs_of_all_paths_on_one_workspace():
    """Captured steps by rows, on codes and on expanded keys, in turn on one workspace; and two streams with a
    workspace each at once."""
    shapes = [([(1, 900), (1, 40)], 0), ([(60, 300), (3, 3), (1, 50)], LONG), ([(90, 300), (70, 70)], 0)]
    ts = [Batch(lens, 8, 2, 128, 16, BF16, seed=20 + i, norm=True, rotary=128, max_len=m) for i, (lens, m) in enumerate(shapes)]
    for t in ts:
        t.args()
    ws = max((t.ws for t in ts), key=lambda w: w.numel())
    own = [t.ws for t in ts]
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for t in ts:
            t.ws = ws
            args = t.args()
            gqaw.check(gqaw.gqaw_paged_i4_step(args, side.cuda_stream))
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                gqaw.check(gqaw.gqaw_paged_i4_step(args, torch.cuda.current_stream().cuda_stream))
            graphs.append((g, args))
        for _ in range(3):
            for (g, _), t in zip(graphs, ts):
                t.out.fill_(7.0)
                g.replay()
        side.synchronize()
    for t in ts:
        t.check_output(turned=True)
    firsts = [t.out.clone() for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    calls = []
    for t, w in zip(ts, own):
        t.ws = w
        t.out.fill_(7.0)
        calls.append(t.args())
    torch.cuda.synchronize()
    for _ in range(3):
        for a, st in zip(calls, streams):
            gqaw.check(gqaw.gqaw_paged_i4_step(a, st.cuda_stream))
    torch.cuda.synchronize()
    for t, first in zip(ts, firsts):
        assert torch.equal(t.out, first)


def test_no_pages_and_no_tokens():
    t = Batch([(0, 0), (0, 0)], 4, 2, 64, 16, BF16, extra_rows=4, spare_pages=1)
    for fn in (gqaw.gqaw_paged_i4_append, gqaw.gqaw_paged_i4_attend, gqaw.gqaw_paged_i4_step, gqaw.gqaw_paged_i4_read):
        t.call(fn)
    assert (t.out == 7.0).all() and (t.ko == 7.0).all()


def test_more_sequences_than_one_launch_takes():
    lens = [(1 + i % 3, 20 + i % 50) for i in range(600)]
    t = Batch(lens, 4, 2, 64, 16, BF16, seed=14)
    t.call(gqaw.gqaw_paged_i4_attend)
    t.check_output()


def test_position_outside_the_tables():
    t = Batch([(2, 40), (1, 30)], 4, 2, 64, 16, BF16, seed=15, rotary=64, position_ids=True)
    t.ids[1] = 10 ** 9
    t.call(gqaw.gqaw_paged_i4_step, flags=gqaw.GQAW_DEV_BAD_POSITION)


def test_graph_replays_and_shared_workspace():
    """Two captured steps of different shapes on one workspace, replayed in turn, on a stream of their own."""
    a = Batch([(1, 900), (1, 40)], 8, 2, 128, 16, BF16, seed=16, norm=True, rotary=128)
    b = Batch([(40, 300), (3, 3)], 8, 2, 128, 16, BF16, seed=17, norm=True, rotary=128)
    a.args(), b.args()
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.ws = b.ws = ws
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for t in (a, b):
            args = t.args()
            gqaw.check(gqaw.gqaw_paged_i4_step(args, side.cuda_stream))
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                gqaw.check(gqaw.gqaw_paged_i4_step(args, torch.cuda.current_stream().cuda_stream))
            graphs.append((g, args))
        for _ in range(3):
            for (g, _), t in zip(graphs, (a, b)):
                t.out.fill_(7.0)
                g.replay()
        side.synchronize()
    for t in (a, b):
        t.check_output(turned=True)
    first = a.out.clone()
    a.call(gqaw.gqaw_paged_i4_step)
    assert torch.equal(first, a.out)


def test_same_inputs_same_bits():
    t = Batch([(1, 5000), (1, 3000), (9, 2000)], 8, 2, 128, 16, BF16, seed=18)
    t.call(gqaw.gqaw_paged_i4_attend)
    first = t.out.clone()
    for _ in range(4):
        t.out.fill_(7.0)
        t.call(gqaw.gqaw_paged_i4_attend)
        assert torch.equal(first, t.out)
