"""The paged operators and the norms without a GPU: what the host refuses, before anything is
enqueued, and what the plan sizes."""
from __future__ import annotations

import ctypes

import pytest
import torch

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from sliding_window_gqa_02_gb300 import build, gqaw

    build.build()
    return gqaw


def _paged(lib, **over):
    """Fake, disjoint, 16-byte-aligned addresses 16 MiB apart: no call here reaches a device."""
    a = lib.gqaw_paged_args()
    base = dict(batch_size=3, total_new_tokens=10, max_new_tokens=6, max_sequence_length=200, num_heads=8,
                kv_num_heads=2, head_size=64, page_size=16, num_pages=40, page_table_width=13, dtype=lib.GQAW_BF16)
    for i, n in enumerate(["query", "key", "value", "output", "key_pages", "value_pages", "page_table", "query_start",
                           "seqlens_k", "workspace"]):
        base[n] = 16 * MB * (i + 1)
    base["workspace_bytes"] = 1 << 30
    base["workspace"] = 1 << 40
    base.update(over)
    for k, v in base.items():
        setattr(a, k, v)
    return a


BAD = [
    (dict(batch_size=-1), 1, "batch_size"),
    (dict(total_new_tokens=-1), 1, "total_new_tokens"),
    (dict(max_new_tokens=11), 1, "max_new_tokens"),
    (dict(max_new_tokens=-1), 1, "max_new_tokens"),
    (dict(num_heads=0), 1, "num_heads"),
    (dict(num_heads=9), 1, "multiple"),
    (dict(dtype=2), 1, "dtype"),
    (dict(head_size=0), 1, "head_size"),
    (dict(head_size=96), 2, "head_size 96"),
    (dict(page_size=0), 1, "page_size"),
    (dict(num_pages=-1), 1, "num_pages"),
    (dict(page_table_width=-1), 1, "page_table_width"),
    (dict(max_sequence_length=5), 1, "max_sequence_length"),
    (dict(max_sequence_length=209), 1, "page_table_width 13"),
    (dict(local_window_size=-1), 1, "local_window_size"),
    (dict(scale=-1.0), 1, "scale"),
    (dict(scale=float("nan")), 1, "scale"),
    (dict(softcap=float("inf")), 1, "softcap"),
    (dict(norm_eps=-1.0), 1, "norm_eps"),
    (dict(reserved=1), 1, "reserved"),
    (dict(num_heads=40000, kv_num_heads=40000), 2, "num_heads"),
    (dict(total_new_tokens=1 << 30), 2, "rows"),
    (dict(query_stride=511), 1, "query_stride"),
    (dict(key_stride=132), 1, "key_stride 132 is not a multiple"),
    (dict(value_stride=-1), 1, "value_stride"),
    (dict(output_stride=1 << 50), 2, "output_stride"),
    (dict(page_stride=2048, head_stride=1024), 1, "all 0"),
    (dict(page_stride=2048, head_stride=1000, row_stride=64), 1, "overlap"),
    (dict(page_stride=2052, head_stride=1024, row_stride=64), 1, "multiple of 16"),
    (dict(page_stride=1024, head_stride=1024, row_stride=64), 1, "overlap"),
    (dict(cos_cache=1 << 41), 1, "go together"),
    (dict(cos_cache=1 << 41, sin_cache=1 << 42, rotary_dim=7, rotary_cache_len=9), 1, "rotary_dim"),
    (dict(cos_cache=1 << 41, sin_cache=1 << 42, rotary_dim=66, rotary_cache_len=9), 1, "rotary_dim"),
    (dict(cos_cache=1 << 41, sin_cache=1 << 42), 1, "rotary_cache_len"),
    (dict(workspace=None), 4, "workspace is NULL"),
    (dict(workspace=(1 << 40) + 64), 4, "256-byte"),
    (dict(workspace_bytes=1000), 4, "workspace_bytes"),
    (dict(query_start=None), 1, "query_start"),
    (dict(seqlens_k=16 * MB + 2), 1, "seqlens_k"),
    (dict(page_table=None), 1, "page_table"),
    (dict(key_pages=None), 1, "key_pages"),
    (dict(value_pages=16 * MB * 6 + 8), 1, "value_pages is not 16-byte"),
    (dict(value_pages=16 * MB * 5), 1, "overlaps"),
    (dict(query_weight=16 * MB * 30 + 8), 1, "weight"),
    (dict(head_sink=16 * MB * 30 + 2), 1, "head_sink"),
]


@pytest.mark.parametrize("over,status,msg", BAD, ids=[str(b[0])[:60] for b in BAD])
def test_paged_refusals(lib, over, status, msg):
    a = _paged(lib, **over)
    seen = 0
    for fn in (lib.gqaw_paged_append, lib.gqaw_paged_attend, lib.gqaw_paged_step):
        if msg == "overlaps" and fn is lib.gqaw_paged_attend:
            continue  # an attention only reads the pages
        assert fn(a, 0) == status
        assert msg in lib.gqaw_last_error(), lib.gqaw_last_error()
        seen += 1
    assert seen


def test_paged_refusals_of_one_call(lib):
    for over, fns, msg in [
        (dict(query=None), ("gqaw_paged_attend", "gqaw_paged_step"), "query is NULL"),
        (dict(output=16 * MB + 8), ("gqaw_paged_attend", "gqaw_paged_step"), "output is not 16-byte"),
        (dict(key=None), ("gqaw_paged_append", "gqaw_paged_step"), "key is NULL"),
        (dict(value=16 * MB + 4), ("gqaw_paged_append", "gqaw_paged_step"), "value is not 16-byte"),
        (dict(output=16 * MB), ("gqaw_paged_attend", "gqaw_paged_step"), "output overlaps query"),
        (dict(key=16 * MB * 5), ("gqaw_paged_append", "gqaw_paged_step"), "key_pages overlaps key"),
        (dict(output=16 * MB * 6), ("gqaw_paged_attend", "gqaw_paged_step"), "output overlaps value_pages"),
        (dict(query=1 << 40), ("gqaw_paged_attend", "gqaw_paged_step"), "workspace overlaps query"),
        (dict(cos_cache=(1 << 41) + 1, sin_cache=1 << 42, rotary_cache_len=9), ("gqaw_paged_append", "gqaw_paged_step"), "cos_cache"),
        (dict(cos_cache=1 << 41, sin_cache=1 << 42, rotary_cache_len=9, position_ids=4), ("gqaw_paged_append", "gqaw_paged_step"),
         "position_ids"),
    ]:
        for fn in fns:
            assert getattr(lib, fn)(_paged(lib, **over), 0) == 1, over
            assert msg in lib.gqaw_last_error(), (over, lib.gqaw_last_error())


def test_nothing_to_do_needs_no_pointers(lib):
    before = lib.gqaw_launch_count()
    for over in (dict(batch_size=0), dict(total_new_tokens=0, max_new_tokens=0), dict(max_new_tokens=0)):
        a = _paged(lib, **over)
        for n in ("query", "key", "value", "output", "key_pages", "value_pages", "page_table", "query_start", "seqlens_k",
                  "workspace"):
            setattr(a, n, None)
        for fn in (lib.gqaw_paged_append, lib.gqaw_paged_attend, lib.gqaw_paged_step):
            assert fn(a, 0) == lib.GQAW_OK
    q = lib.gqaw_qk_args()
    q.head_size, q.num_heads = 64, 2
    assert lib.gqaw_qk_norm_rotary(q, 0) == lib.GQAW_OK
    assert lib.gqaw_launch_count() == before


def test_paged_workspace(lib):
    """The split results follow the grid, the turned queries (two parts of bf16) the tokens; sizes alone matter."""
    a = _paged(lib, query=None, workspace=None)
    n = lib.gqaw_paged_workspace_bytes(a)
    assert n > 4096 and n % 256 == 0
    more = lib.gqaw_paged_workspace_bytes(_paged(lib, total_new_tokens=1010))
    assert more - n == 2 * ((1010 * 8 * 64 * 2 + 255) // 256 * 256 - 10 * 8 * 64 * 2 // 256 * 256)
    assert lib.gqaw_paged_workspace_bytes(_paged(lib, batch_size=3000)) < n + 64 * MB
    assert lib.gqaw_paged_workspace_bytes(_paged(lib, head_size=96)) == 0


def _qk(lib, **over):
    a = lib.gqaw_qk_args()
    base = dict(num_tokens=10, num_heads=8, kv_num_heads=2, head_size=64, dtype=lib.GQAW_F32, norm_eps=1e-6)
    for i, n in enumerate(["query", "key", "query_out", "key_out"]):
        base[n] = 16 * MB * (i + 1)
    base.update(over)
    for k, v in base.items():
        setattr(a, k, v)
    return a


ROT = dict(cos_cache=1 << 41, sin_cache=1 << 42, rotary_cache_len=9)


@pytest.mark.parametrize("over,status,msg", [
    (dict(num_tokens=-1), 1, "num_tokens"),
    (dict(num_heads=-1), 1, "num_heads"),
    (dict(dtype=3), 1, "dtype"),
    (dict(head_size=80), 2, "head_size 80"),
    (dict(norm_eps=float("nan")), 1, "norm_eps"),
    (dict(reserved=2), 1, "reserved"),
    (dict(num_heads=70000), 2, "heads"),
    (dict(num_tokens=1 << 30), 2, "rows"),
    (dict(query_stride=100), 1, "query_stride"),
    (dict(key_out_stride=130), 1, "key_out_stride 130"),
    (dict(query=None), 1, "query is NULL"),
    (dict(key_out=16 * MB + 4), 1, "key_out is not 16-byte"),
    (dict(query_out=16 * MB + 1024), 1, "query_out overlaps query"),
    (dict(query_out=16 * MB, query_out_stride=1024), 1, "query_out overlaps query"),
    (dict(key_out=16 * MB * 3), 1, "overlaps"),
    (dict(key_out=16 * MB), 1, "key_out overlaps query"),
    (dict(query_weight=8), 1, "weight"),
    (dict(cos_cache=1 << 41), 1, "go together"),
    (dict(ROT, rotary_dim=3), 1, "rotary_dim"),
    (dict(ROT, rotary_cache_len=0), 1, "rotary_cache_len"),
    (dict(ROT), 1, "position_ids is NULL"),
    (dict(ROT, position_ids=4), 1, "position_ids"),
    (dict(ROT, position_ids=1 << 43), 4, "workspace is NULL"),
    (dict(ROT, position_ids=1 << 43, workspace=1 << 44, workspace_bytes=100), 4, "workspace_bytes"),
])
def test_qk_refusals(lib, over, status, msg):
    assert lib.gqaw_qk_norm_rotary(_qk(lib, **over), 0) == status
    assert msg in lib.gqaw_last_error(), lib.gqaw_last_error()


def test_struct_sizes(lib):
    assert lib.load().gqaw_qk_args_size() == ctypes.sizeof(lib.gqaw_qk_args)
    assert lib.load().gqaw_paged_args_size() == ctypes.sizeof(lib.gqaw_paged_args)


def test_binding_checks_shapes(lib):
    """make_paged_args and make_qk_args refuse tensors that do not fit together (CPU tensors:
    nothing is called with them)."""
    D, Nq, Nkv, page = 64, 4, 2, 16
    t = dict(query=torch.zeros(5, Nq * D), key=torch.zeros(5, Nkv * D), value=torch.zeros(5, Nkv, D),
             key_pages=torch.zeros(7, Nkv, page, D), value_pages=torch.zeros(7, Nkv, page, D),
             page_table=torch.zeros(3, 4, dtype=torch.int32), query_start=torch.zeros(4, dtype=torch.int32),
             seqlens_k=torch.zeros(3, dtype=torch.int32), max_new_tokens=2, max_sequence_length=64, num_heads=Nq,
             kv_num_heads=Nkv, output=torch.zeros(5, Nq * D))
    a = lib.make_paged_args(**t)
    assert (a.batch_size, a.total_new_tokens, a.page_size, a.num_pages, a.page_table_width) == (3, 5, page, 7, 4)
    assert (a.page_stride, a.head_stride, a.row_stride) == (Nkv * page * D, page * D, D)
    hir = dict(t, key_pages=torch.zeros(7, page, Nkv, D), value_pages=torch.zeros(7, page, Nkv, D), heads_inside_rows=True)
    a = lib.make_paged_args(**hir)
    assert (a.page_size, a.page_stride, a.head_stride, a.row_stride) == (page, page * Nkv * D, D, Nkv * D)
    both = torch.zeros(7, 2, Nkv, page, D)
    a = lib.make_paged_args(**dict(t, key_pages=both[:, 0], value_pages=both[:, 1]))
    assert a.page_stride == 2 * Nkv * page * D
    wide = torch.zeros(5, (Nq + 2 * Nkv) * D)
    a = lib.make_paged_args(**dict(t, query=wide[:, :Nq * D], key=wide[:, Nq * D:(Nq + Nkv) * D]))
    assert a.query_stride == a.key_stride == (Nq + 2 * Nkv) * D
    for bad in (dict(query=torch.zeros(4, Nq * D)), dict(query=torch.zeros(5, Nq * D + 1)),
                dict(query=torch.zeros(5, Nq * D, dtype=torch.bfloat16)), dict(key=torch.zeros(Nkv * D, 5).T),
                dict(value_pages=torch.zeros(7, Nkv, page, 2 * D)[..., :D]), dict(kv_num_heads=4),
                dict(page_table=torch.zeros(3, 4)), dict(page_table=torch.zeros(3, 8, dtype=torch.int32)[:, ::2]),
                dict(query_start=torch.zeros(3, dtype=torch.int32)), dict(seqlens_k=torch.zeros(3, dtype=torch.int64)),
                dict(head_sink=torch.zeros(Nkv)), dict(query_weight=torch.zeros(D + 1)),
                dict(cos_cache=torch.zeros(9, 32)), dict(cos_cache=torch.zeros(9, 32), sin_cache=torch.zeros(9, 16)),
                dict(position_ids=torch.zeros(4, dtype=torch.int64)),
                dict(value=torch.zeros(5, D, Nkv).transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            lib.make_paged_args(**dict(t, **bad))
    q = dict(query=t["query"], key=t["key"], query_out=torch.zeros(5, Nq * D), key_out=torch.zeros(5, Nkv * D),
             num_heads=Nq, kv_num_heads=Nkv, head_size=D)
    assert lib.make_qk_args(**q).num_tokens == 5
    for bad in (dict(key_out=torch.zeros(6, Nkv * D)), dict(query=None, key=None), dict(query_weight=torch.zeros(3)),
                dict(position_ids=torch.zeros(5)), dict(key=torch.zeros(5, Nkv * D, dtype=torch.bfloat16))):
        with pytest.raises((ValueError, TypeError)):
            lib.make_qk_args(**dict(q, **bad))


def test_binding_refuses_overlapping_rows_and_foreign_workspaces(lib):
    """A stride of 0 means contiguous rows to the library: an expanded tensor is refused before that."""
    one = torch.zeros(1, 4 * 16)
    rows, kv, pages = torch.zeros(5, 4 * 16), torch.zeros(5, 2 * 16), torch.zeros(3, 2, 8, 16)
    table, start, lens = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)

    def paged(q=rows, k=kv, kp=pages, **kw):
        return lib.make_paged_args(q, k, kv, kp, kp, table, start, lens, 5, 24, 4, 2, rows, **kw)

    paged()
    for kw in (dict(q=one.expand(5, -1)), dict(k=torch.zeros(5 * 32).as_strided((5, 32), (16, 1))),
               dict(kp=torch.zeros(1, 1, 1, 16).expand(3, 2, 8, 16)), dict(kp=torch.zeros(1, 2, 8, 16).expand(3, 2, 8, 16)),
               dict(workspace=torch.zeros(4096, dtype=torch.uint8, device="meta")),
               dict(workspace=torch.zeros(8192, dtype=torch.uint8)[::2])):
        with pytest.raises(ValueError):
            paged(**kw)
    lib.make_qk_args(rows, None, rows, None, 4, 0, 16)
    for q, kw in ((one.expand(5, -1), {}), (rows, dict(workspace=torch.zeros(256, dtype=torch.uint8, device="meta")))):
        with pytest.raises(ValueError):
            lib.make_qk_args(q, None, rows, None, 4, 0, 16, **kw)
