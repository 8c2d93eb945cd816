"""gqaw_qk_norm_rotary on a GB300 against the 64-bit definition."""
from __future__ import annotations

import pytest
import torch

import paged_reference as ref
from sliding_window_gqa_02_gb300 import gqaw

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _tables(rows, rd, dtype):
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)
    return torch.cos(ang).to(dtype).cuda().contiguous(), torch.sin(ang).to(dtype).cuda().contiguous()


def _run(N, Nq, Nkv, D, dtype, rd, interleaved, norm, in_place=False, fused=False, eps=1e-6, table_shift=0, bad=None,
         scale=1.0):
    g = torch.Generator().manual_seed(N * 31 + D)
    if fused:
        x = (torch.randn(N, (Nq + Nkv + 1) * D, generator=g) * scale).to(dtype).cuda()
        q, k = x[:, :Nq * D], x[:, Nq * D:(Nq + Nkv) * D]
    else:
        q, k = ((torch.randn(N, h * D, generator=g) * scale).to(dtype).cuda() for h in (Nq, Nkv))
    qw, kw = ((1 + torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)) if norm else (None, None)
    cos = sin = ids = None
    rows = 400
    if rd:
        cos, sin = _tables(rows, rd, dtype)
        if table_shift:
            flat = [torch.empty(t.numel() + table_shift, dtype=dtype, device="cuda") for t in (cos, sin)]
            for f, t in zip(flat, (cos, sin)):
                f[table_shift:] = t.flatten()
            cos, sin = (f[table_shift:].view(rows, rd // 2) for f in flat)
        ids = torch.randint(0, rows, (N,), generator=g).cuda()
        if bad is not None:
            ids[N // 2] = bad
    want = []
    for t, w, h in ((q, qw, Nq), (k, kw, Nkv)):
        want.append(ref.norm_turn(t.reshape(-1, h, D).clone(), w, eps, cos, sin, ids.clamp(0, rows - 1) if rd else None,
                                  interleaved))
    rest = x[:, (Nq + Nkv) * D:].clone() if fused else None
    qo, ko = (q, k) if in_place else (torch.full_like(q, 7), torch.full_like(k, 7))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    a = gqaw.make_qk_args(q, k, qo, ko, Nq, Nkv, D, query_weight=qw, key_weight=kw, norm_eps=eps, cos_cache=cos,
                          sin_cache=sin, position_ids=ids, rotary_interleaved=interleaved, workspace=ws)
    gqaw.check(gqaw.gqaw_qk_norm_rotary(a, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    _, flags = gqaw.gqaw_device_status(ws.data_ptr(), stream=torch.cuda.current_stream().cuda_stream)
    assert flags == (gqaw.GQAW_DEV_BAD_POSITION if bad is not None else 0)
    for t, (w, bound), h in ((qo, want[0], Nq), (ko, want[1], Nkv)):
        got = t.reshape(-1, h, D).double()
        tol = bound + ref.u(dtype) * (w.abs() + bound)
        ok = (got - w).abs() <= tol
        if bad is not None:
            ok[N // 2] = True
        assert ok.all(), float(((got - w).abs() - tol).max())
    if rest is not None:
        assert torch.equal(x[:, (Nq + Nkv) * D:], rest)
    return qo, ko


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(dtype, D, interleaved):
    for N, Nq, Nkv in ((1, 1, 1), (3, 7, 1), (65, 12, 4)):
        _run(N, Nq, Nkv, D, dtype, D, interleaved, True)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rd", [0, 2, 6, 16, 20, 32, 62])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary_widths(dtype, rd, norm):
    for interleaved in (False, True):
        _run(37, 6, 2, 64, dtype, rd, interleaved, norm)
        if rd:
            _run(37, 6, 2, 64, dtype, rd, interleaved, norm, table_shift=1)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("in_place", [False, True])
def test_slices_and_in_place(dtype, in_place):
    _run(50, 8, 2, 128, dtype, 128, False, True, in_place=in_place, fused=True)
    _run(50, 8, 2, 64, dtype, 12, False, True, in_place=in_place)


@pytest.mark.parametrize("dtype", [BF, F])
def test_one_side_only(dtype):
    x = torch.randn(9, 4 * 64, device="cuda").to(dtype)
    w = torch.ones(64, dtype=dtype, device="cuda")
    q, k = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.current_stream().cuda_stream
    gqaw.check(gqaw.gqaw_qk_norm_rotary(gqaw.make_qk_args(x, None, q, None, 4, 0, 64, query_weight=w), s))
    gqaw.check(gqaw.gqaw_qk_norm_rotary(gqaw.make_qk_args(None, x, None, k, 0, 4, 64, key_weight=w), s))
    assert torch.equal(q, k)


def test_small_and_large_rows():
    """Rows whose mean square the epsilon drowns, zero rows, and rows of 10^15."""
    for dtype in (BF, F):
        _run(5, 2, 1, 64, dtype, 64, False, True, scale=1e-6, eps=1e-5)
        _run(5, 2, 1, 64, dtype, 64, False, True, scale=1e15)
        q, k = _run(5, 2, 1, 64, dtype, 64, True, True, scale=0.0)
        assert (q == 0).all() and (k == 0).all()


@pytest.mark.parametrize("bad", [-1, 400, 1 << 40])
def test_bad_position(bad):
    _run(21, 4, 2, 128, BF, 128, False, True, bad=bad)


def test_no_rotation_is_a_plain_step_input():
    """Without weights and tables the rows pass through bit for bit."""
    x = torch.randn(7, 6 * 32, device="cuda")
    o = torch.empty_like(x)
    s = torch.cuda.current_stream().cuda_stream
    gqaw.check(gqaw.gqaw_qk_norm_rotary(gqaw.make_qk_args(x, None, o, None, 6, 0, 32), s))
    assert torch.equal(x, o)


def test_graph_replay_reads_new_inputs():
    x = torch.randn(64, 8 * 128, device="cuda").to(BF)
    w = torch.ones(128, dtype=BF, device="cuda")
    o = torch.empty_like(x)
    a = gqaw.make_qk_args(x, None, o, None, 8, 0, 128, query_weight=w)
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        gqaw.check(gqaw.gqaw_qk_norm_rotary(a, st.cuda_stream))
    x.mul_(-2)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want, bound = ref.norm_turn(x.view(64, 8, 128), w, 1e-6, None, None, None, False)
    assert ((o.view(64, 8, 128).double() - want).abs() <= bound + ref.u(BF) * want.abs() * (1 + 1e-3)).all()
