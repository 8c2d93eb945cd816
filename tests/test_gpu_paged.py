"""Paged attention, paged append and the paged step on a GB300, against the 64-bit definition.

Unowned pages and rows past a sequence's length hold NaN throughout, and table entries that no
token needs are out of range, so a read past what the definition allows shows up.
"""
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


RAGGED = [(1, 1), (1, 131), (0, 0), (1, 127), (1, 128), (0, 40), (1, 129), (1, 700)]
CHUNKS = [(5, 5), (40, 300), (0, 0), (1, 260), (129, 129), (64, 517), (0, 33), (3, 128)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens", [[(1, 1)], RAGGED, CHUNKS], ids=["one", "decode", "chunks"])
@pytest.mark.parametrize("D,Nq,Nkv,page", [(64, 8, 2, 16), (128, 8, 2, 16), (128, 4, 4, 128), (128, 7, 1, 32),
                                           (64, 10, 2, 64), (256, 6, 2, 16), (128, 32, 2, 8), (32, 4, 2, 16),
                                           (8, 2, 1, 4), (16, 6, 2, 24), (128, 4, 1, 1), (64, 4, 2, 256)])
def test_attend(dtype, lens, D, Nq, Nkv, page):
    b = Batch(lens, Nq, Nkv, D, page, dtype, seed=1, extra_rows=3, lead_rows=2)
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()
    b.check_untouched()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens", [RAGGED, [(8, 70), (5, 900), (8, 8), (2, 333)], CHUNKS], ids=["decode", "verify", "chunks"])
@pytest.mark.parametrize("window", [1, 37, 128, 300, 5000])
def test_window(dtype, lens, window):
    b = Batch(lens, 8, 2, 128, 16, dtype, seed=2, window=window)
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()


MIXED = [(1, 500), (2, 300), (1, 1), (70, 200), (0, 9), (3, 4), (1, 129), (8, 2000), (9, 9), (2, 2), (140, 141)]


@pytest.mark.parametrize("kw", [dict(), dict(window=100, sink=True), dict(softcap=20.0)], ids=str)
@pytest.mark.parametrize("D,Nq,Nkv,page,launches", [(64, 16, 16, 16, 2), (64, 64, 8, 64, 2), (128, 32, 8, 32, 2), (128, 24, 8, 16, 2),
                                                    (128, 8, 2, 32, 1), (256, 32, 8, 16, 1), (128, 72, 8, 16, 1)])
def test_short_sequences_among_chunks(D, Nq, Nkv, page, launches, kw):
    """Many sequences of a few rows take the kernel for few rows, in a launch of their own: every
    sequence is one launch's, on either side of the border of 8 rows."""
    b = Batch(MIXED, Nq, Nkv, D, page, BF, seed=21, extra_rows=2, **kw)
    n0 = gqaw.gqaw_launch_count()
    b.call(gqaw.gqaw_paged_attend)
    assert gqaw.gqaw_launch_count() - n0 == launches
    b.check_output()
    b.check_untouched()
    first = b.out.clone()
    b.call(gqaw.gqaw_paged_attend)  # the workspace as the launches left it
    assert torch.equal(first, b.out)


def test_equal_chunks_are_one_launch():
    b = Batch([(9, 300)] * 4, 8, 2, 64, 16, BF, seed=22)
    n0 = gqaw.gqaw_launch_count()
    b.call(gqaw.gqaw_paged_attend)
    assert gqaw.gqaw_launch_count() - n0 == 1
    b.check_output()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("kw", [dict(softcap=20.0), dict(sink=True), dict(smooth=True), dict(scale=0.31),
                                dict(softcap=5.0, sink=True, window=50)], ids=str)
@pytest.mark.parametrize("lens", [RAGGED, CHUNKS], ids=["decode", "chunks"])
def test_options(dtype, kw, lens):
    b = Batch(lens, 8, 2, 64, 32, dtype, seed=3, **kw)
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens", [RAGGED, CHUNKS], ids=["decode", "chunks"])
@pytest.mark.parametrize("D", [64, 128])
def test_layouts_and_strides(dtype, lens, D):
    """Heads inside rows, query and output as slices of wider tensors."""
    b = Batch(lens, 8, 2, D, 16, dtype, seed=4, heads_inside_rows=True, fused=True)
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()
    wide = torch.full((b.out.shape[0], 10 * D), 7.0, dtype=dtype, device="cuda")
    plain = b.out.clone()
    b.out = wide[:, D:9 * D]
    b.call(gqaw.gqaw_paged_attend)
    assert torch.equal(b.out, plain)
    assert (wide[:, :D] == 7).all() and (wide[:, 9 * D:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(1, 9000), (1, 40), (1, 20000)], [(8, 9000), (3, 16000)], [(4, 9000), (1, 9999)],
                                  [(16, 9000), (300, 6000)]], ids=["decode", "verify8", "verify4", "chunks"])
def test_long_split(dtype, lens, D):
    """Few sequences, long axes: units cut over many CTAs and merged, rings that go round often."""
    b = Batch(lens, 4, 1, D, 64, dtype, seed=5)
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()
    again = b.out.clone()
    b.out.fill_(7.0)
    b.call(gqaw.gqaw_paged_attend)
    assert torch.equal(b.out, again)  # the merge order does not depend on which CTA is last


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("S", [4, 60])
@pytest.mark.parametrize("window", [0, 20])
def test_non_finite_rows_reach_only_who_attends_them(dtype, value, S, window):
    """A non-finite value (and key) row inside the sequence spoils the tokens that attend it
    and no other."""
    T = 200
    b = Batch([(S, T), (1, 77)], 8, 2, 128, 16, dtype, seed=6, window=window)
    for j in (T - S + 2, T - 2):
        b.vp[int(b.table[0, j // 16]), :, j % 16, 5::7] = value
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()
    b2 = Batch([(S, T), (1, 77)], 8, 2, 128, 16, dtype, seed=6, window=window)
    j = T - S + 2
    b2.kp[int(b2.table[0, j // 16]), :, j % 16] = float("nan")
    b2.call(gqaw.gqaw_paged_attend)
    rows = b2.out[b2.rows(0)].reshape(S, -1)
    seen = torch.tensor([s >= 2 and (not window or s - 2 < window) for s in range(S)], device="cuda")
    assert torch.isnan(rows[seen]).all() and torch.isfinite(rows[~seen]).all()


@pytest.mark.parametrize("dtype", [BF, F])
def test_large_logits(dtype):
    """Logits far apart (maxima that move by hundreds from tile to tile) and far below zero."""
    b = Batch([(1, 1000), (9, 640), (200, 400)], 4, 2, 128, 16, dtype, seed=7, scale=2.0)
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()
    b.kp *= torch.where(torch.isnan(b.kp), b.kp, torch.full_like(b.kp, 4.0))
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("S", [1, 3, 50, 90])
def test_many_sequences(dtype, S):
    """More sequences than one launch takes, most of them idle."""
    lens = [(0, 0) if i % 3 else (min(S, 1 + i % 90), 1 + i % 90) for i in range(700)]
    b = Batch(lens, 4, 2, 64, 16, dtype, seed=8)
    b.call(gqaw.gqaw_paged_attend)
    b.check_output()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens", [RAGGED, CHUNKS], ids=["decode", "chunks"])
@pytest.mark.parametrize("D,page,hir", [(128, 16, False), (64, 32, True), (256, 8, False), (32, 5, False), (8, 16, True)])
@pytest.mark.parametrize("norm,rotary,interleaved", [(False, 0, False), (True, 1.0, False), (True, 1.0, True),
                                                     (False, 0.5, False), (True, 0, False), (False, 0.25, True)])
def test_append(dtype, lens, D, page, hir, norm, rotary, interleaved):
    rd = int(rotary * D)
    b = Batch(lens, 4, 2, D, page, dtype, seed=9, heads_inside_rows=hir, norm=norm, rotary=rd, interleaved=interleaved,
              filled=False, extra_rows=2, lead_rows=1, fused=True, position_ids=interleaved and norm)
    k0, v0 = b.kp.clone(), b.vp.clone()
    b.call(gqaw.gqaw_paged_append)
    b.check_pages(k0, v0)


@pytest.mark.parametrize("rd", [2, 12, 28, 60])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_odd_rotary_widths(rd, interleaved):
    b = Batch([(3, 9), (2, 2)], 6, 3, 64, 16, BF, seed=10, norm=True, rotary=rd, interleaved=interleaved, filled=False)
    k0, v0 = b.kp.clone(), b.vp.clone()
    b.call(gqaw.gqaw_paged_append)
    b.check_pages(k0, v0)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens", [RAGGED, [(8, 70), (5, 900), (8, 8)], CHUNKS], ids=["decode", "verify", "chunks"])
@pytest.mark.parametrize("D,kw", [(128, dict(norm=True, rotary=128)), (64, dict(rotary=32, interleaved=True, window=50)),
                                  (128, dict()), (256, dict(norm=True, rotary=256, softcap=15.0))], ids=str)
def test_step(dtype, lens, D, kw):
    """The step against the definition, and against its three parts one after the other: the same
    bits, but where bf16 queries turned by the step keep a second part that the parts' do not."""
    two = dtype == BF and "rotary" in kw
    mk = lambda: Batch(lens, 8, 2, D, 16, dtype, seed=11, filled=False, extra_rows=1, **kw)
    b = mk()
    k0, v0 = b.kp.clone(), b.vp.clone()
    b.call(gqaw.gqaw_paged_step)
    b.check_pages(k0, v0)
    b.check_output(turned=True, parts=2 if two else 1)
    b.check_untouched()
    c = mk()
    c.call(gqaw.gqaw_paged_append)
    if c.qw is not None or c.cos is not None:
        q = torch.empty_like(c.q)
        a = gqaw.make_qk_args(c.q, None, q, None, c.Nq, 0, D, query_weight=c.qw, norm_eps=1e-5, cos_cache=c.cos,
                              sin_cache=c.sin, position_ids=c.pos.cuda() if c.cos is not None else None,
                              rotary_interleaved=c.interleaved, workspace=c.ws)
        gqaw.check(gqaw.gqaw_qk_norm_rotary(a, torch.cuda.current_stream().cuda_stream))
        c.q = q
    c.call(gqaw.gqaw_paged_attend)
    if two:
        c.check_output()
    else:
        assert torch.equal(b.out, c.out)
    assert torch.equal(torch.nan_to_num(b.kp), torch.nan_to_num(c.kp))


@pytest.mark.parametrize("dtype", [BF, F])
def test_sequence_of_steps(dtype):
    """A prompt, a verify step and single tokens through one workspace: each against the
    definition over what the cache then holds, and against gqa_windowed_step over the same
    tokens with the same window."""
    Nq, Nkv, D, page, W = 8, 2, 128, 16, 48
    steps = [70, 5, 1, 1, 33, 1]
    ws, T = None, 0
    C = 64
    dev = "cuda"
    pk = torch.zeros(1, Nkv, C, D, dtype=dtype, device=dev)
    pv = torch.zeros_like(pk)
    total = sum(steps)
    pages = total // page + 1
    kp, vp = (torch.full((pages, Nkv, page, D), float("nan"), dtype=dtype, device=dev) for _ in range(2))
    table = torch.randperm(pages).to(torch.int32)[None].cuda()
    for n, S in enumerate(steps):
        T += S
        b = Batch([(S, T)], Nq, Nkv, D, page, dtype, seed=20 + n, window=W, filled=False)
        b.kp, b.vp, b.table, b.max_len = kp, vp, table, total
        if ws is None:
            b.max_new, keep = max(steps), b.max_new
            b.q, b.k, b.v, b.out = (torch.zeros(70, x.shape[1], dtype=dtype, device=dev) for x in (b.q, b.k, b.v, b.out))
            b.args()
            ws = b.ws
            b = Batch([(S, T)], Nq, Nkv, D, page, dtype, seed=20 + n, window=W, filled=False)
            b.kp, b.vp, b.table, b.max_len = kp, vp, table, total
        b.ws = ws
        b.call(gqaw.gqaw_paged_step)
        b.check_output()
        out = torch.empty_like(b.out)
        seq = torch.tensor([T - 1], dtype=torch.int32, device=dev)
        mk = lambda w: gqaw.make_args(b.q[None], b.k[None], b.v[None], pk, pv, pk, pv, seq, total, Nq, Nkv, W, out[None],
                                      workspace=w)
        need = gqaw.gqaw_workspace_bytes(mk(None))
        if need > ws.numel():
            w2 = gqaw.new_workspace(mk(None), dev, torch.cuda.current_stream().cuda_stream)
        else:
            w2 = ws  # the paged and the windowed step share the workspace, in stream order
        gqaw.check(gqaw.gqa_windowed_step(mk(w2), torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        b.out = out
        b.check_output()


@pytest.mark.parametrize("lens", [RAGGED, CHUNKS, [(1, 9000), (1, 30)]], ids=["decode", "chunks", "long"])
def test_bad_page_is_flagged_and_others_are_right(lens):
    for dtype in (BF, F):
        for bad in (-1, 10 ** 6):
            b = Batch(lens, 8, 2, 128, 16, dtype, seed=12)
            b.table[1, 0] = bad
            b.call(gqaw.gqaw_paged_attend, flags=gqaw.GQAW_DEV_BAD_PAGE)
            b.check_output(skip=(1,))
            c = Batch(lens, 8, 2, 128, 16, dtype, seed=12, filled=False)
            j = (c.lens[1][1] - c.lens[1][0]) // 16
            c.table[1, j] = bad
            k0, v0 = c.kp.clone(), c.vp.clone()
            c.call(gqaw.gqaw_paged_append, flags=gqaw.GQAW_DEV_BAD_PAGE)
            c.table[1, j] = -1
            c.check_pages(k0, v0)


@pytest.mark.parametrize("what", ["long", "short", "negative", "past"])
@pytest.mark.parametrize("dtype", [BF, F])
def test_bad_lengths_are_flagged_and_others_are_right(what, dtype):
    b = Batch([(2, 30), (3, 40), (1, 90)], 8, 2, 128, 16, dtype, seed=13, extra_rows=1)
    if what == "long":
        b.seqlens[1] = 1000
    elif what == "short":
        b.seqlens[1] = 1
    elif what == "negative":
        b.starts[1] = 6  # the second sequence runs backwards, the first is longer than any may be
    else:
        b.starts[3] = 50
    skip = {"long": (1,), "short": (1,), "negative": (0, 1), "past": (2,)}[what]
    b.call(gqaw.gqaw_paged_attend, flags=gqaw.GQAW_DEV_BAD_SEQLEN)
    b.check_output(skip=skip)
    b.call(gqaw.gqaw_paged_append, flags=gqaw.GQAW_DEV_BAD_SEQLEN)


@pytest.mark.parametrize("dtype", [BF, F])
def test_graphs_share_a_workspace(dtype):
    """Two captured steps of different shapes on one workspace, replayed in turn, and direct
    calls between them, give the direct calls' bits."""
    a = Batch([(1, 3000), (1, 50)], 8, 2, 128, 16, dtype, seed=14, norm=True, rotary=128, filled=False)
    b = Batch([(60, 2500), (1, 7)], 8, 2, 128, 16, dtype, seed=15, norm=True, rotary=128, filled=False)
    b.args()
    a.args()
    ws = a.ws if a.ws.numel() > b.ws.numel() else b.ws
    a.ws = b.ws = ws
    for x in (a, b):
        x.call(gqaw.gqaw_paged_step)
    want = [x.out.clone() for x in (a, b)]
    stream = torch.cuda.Stream()
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        args = x.args()
        with torch.cuda.graph(g, stream=stream):
            gqaw.check(gqaw.gqaw_paged_step(args, stream.cuda_stream))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1, 0)):
        for i in order:
            (a, b)[i].out.fill_(7.0)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal((a, b)[i].out, want[i])
        a.out.fill_(7.0)
        a.call(gqaw.gqaw_paged_step)
        assert torch.equal(a.out, want[0])


@pytest.mark.parametrize("dtype", [BF, F])
def test_two_streams(dtype):
    """Two calls at once on two streams with a workspace each."""
    bs = [Batch([(1, 4000), (30, 900)], 8, 2, 128, 16, dtype, seed=16 + i) for i in range(2)]
    for b in bs:
        b.call(gqaw.gqaw_paged_attend)
    want = [b.out.clone() for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    args = [b.args() for b in bs]
    for _ in range(20):
        for a, s in zip(args, streams):
            gqaw.check(gqaw.gqaw_paged_attend(a, s.cuda_stream))
    torch.cuda.synchronize()
    for b, w in zip(bs, want):
        assert torch.equal(b.out, w)


@pytest.mark.parametrize("dtype", [BF, F])
def test_offsets_past_32_bits(dtype):
    """A cache whose used pages lie beyond 2^31 elements (and 2^32 bytes)."""
    Nq, Nkv, D, page = 4, 1, 128, 16
    pages = (1 << 31) // (Nkv * page * D) + 64
    kp, vp = (torch.empty(pages, Nkv, page, D, dtype=dtype, device="cuda") for _ in range(2))
    for lens in ([(1, 300), (1, 64)], [(40, 200), (1, 64)]):
        b = Batch(lens, Nq, Nkv, D, page, dtype, seed=18, filled=False)
        small_k, small_v, n = b.kp, b.vp, b.kp.shape[0]
        used = torch.nonzero(b.table >= 0)
        kp[pages - n:], vp[pages - n:] = small_k, small_v
        b.table[b.table >= 0] += pages - n
        b.kp, b.vp = kp, vp
        b.call(gqaw.gqaw_paged_step)
        b.check_output()
        assert used.numel()


def test_host_memory_is_refused():
    """A workspace or query that is not this device's memory is refused before any launch."""
    b = Batch([(1, 40)], 4, 2, 64, 16, BF, seed=23, norm=True, rotary=64)
    a = b.args()
    n0, stream = gqaw.gqaw_launch_count(), torch.cuda.current_stream().cuda_stream
    host = torch.zeros(a.workspace_bytes + 256, dtype=torch.uint8).pin_memory()
    a.workspace = (host.data_ptr() + 255) // 256 * 256
    for fn in (gqaw.gqaw_paged_append, gqaw.gqaw_paged_attend, gqaw.gqaw_paged_step):
        assert fn(a, stream) == gqaw.GQAW_EINVAL
    rows = torch.zeros(3, 4 * 64, dtype=BF).pin_memory()
    q = gqaw.gqaw_qk_args(num_tokens=3, num_heads=4, head_size=64, dtype=gqaw.GQAW_BF16, query=rows.data_ptr(),
                          query_out=rows.data_ptr())
    assert gqaw.gqaw_qk_norm_rotary(q, stream) == gqaw.GQAW_EINVAL
    assert gqaw.gqaw_launch_count() == n0


def test_steps_one_after_the_other_without_waiting():
    """Steps of several shapes enqueued together through one workspace, each reading what the
    one before it appended: the bits of the same steps with a wait between them."""
    outs = []
    for wait in (True, False):
        g = torch.Generator().manual_seed(24)
        Nq, Nkv, D, page = 16, 4, 128, 16
        steps = [300, 1, 7, 1, 90, 1, 1]
        total = sum(steps)
        kp, vp = (torch.zeros(total // page + 1, Nkv, page, D, dtype=BF, device="cuda") for _ in range(2))
        table = torch.randperm(kp.shape[0], generator=g).to(torch.int32)[None].cuda()
        w = (torch.rand(D, generator=g) + 0.5).to(BF).cuda()
        calls, T = [], 0
        for S in steps:
            q, k, v = (torch.randn(S, n * D, generator=g).to(BF).cuda() for n in (Nq, Nkv, Nkv))
            T += S
            calls.append(gqaw.make_paged_args(q, k, v, kp, vp, table, torch.tensor([0, S], dtype=torch.int32, device="cuda"),
                                              torch.tensor([T - 1], dtype=torch.int32, device="cuda"), S, total, Nq, Nkv,
                                              torch.empty_like(q), query_weight=w, key_weight=w))
            calls[-1].keep = (q, k, v)
        size = max(gqaw.gqaw_paged_workspace_bytes(a) for a in calls)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream
        gqaw.check(gqaw.gqaw_workspace_init(ws.data_ptr(), size, stream))
        out = [torch.zeros(S, Nq * D, dtype=BF, device="cuda") for S in steps]
        for a, o in zip(calls, out):
            a.workspace, a.workspace_bytes, a.output = ws.data_ptr(), size, o.data_ptr()
        torch.cuda.synchronize()
        for a in calls:
            gqaw.check(gqaw.gqaw_paged_step(a, stream))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        outs.append(out + [kp])
    for x, y in zip(*outs):
        assert torch.equal(x, y)
