"""The operators on 4-bit caches without a GPU: what the host refuses, and the definition of the codes."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import i4_reference as i4

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from sliding_window_gqa_02_gb300 import build, gqaw

    build.build()
    return gqaw


def _args(lib, **over):
    """Fake, disjoint, 16-byte-aligned addresses 16 MiB apart: no call here reaches a device."""
    x = lib.gqaw_paged_i4_args()
    base = dict(batch_size=3, total_new_tokens=10, max_new_tokens=6, max_sequence_length=200, num_heads=8,
                kv_num_heads=2, head_size=64, page_size=16, num_pages=40, page_table_width=13, dtype=lib.GQAW_BF16)
    names = ["query", "key", "value", "output", "key_pages", "value_pages", "page_table", "query_start", "seqlens_k",
             "key_scales", "value_scales", "key_out", "value_out"]
    for i, n in enumerate(names):
        base[n] = 16 * MB * (i + 1)
    base.update(workspace=1 << 40, workspace_bytes=1 << 30)
    base.update(over)
    own = {f for f, _ in lib.gqaw_paged_i4_args._fields_}
    for k, v in base.items():
        setattr(x if k in own else x.paged, k, v)
    return x


CALLS = ("gqaw_paged_i4_append", "gqaw_paged_i4_attend", "gqaw_paged_i4_step", "gqaw_paged_i4_read")


@pytest.mark.parametrize("over,status,msg", [
    (dict(batch_size=-1), 1, "batch_size"),
    (dict(head_size=16), 2, "4-bit"),
    (dict(head_size=96), 2, "head_size 96"),
    (dict(dtype=2), 1, "dtype"),
    (dict(num_heads=9), 1, "multiple"),
    (dict(reserved=1), 1, "reserved"),
    (dict(max_sequence_length=209), 1, "page_table_width 13"),
    (dict(page_stride=2048, head_stride=512, row_stride=24), 1, "at least 32"),
    (dict(page_stride=2048, head_stride=512, row_stride=40), 1, "multiple of 16"),
    (dict(page_stride=1024, head_stride=496, row_stride=32), 1, "overlap"),
    (dict(page_stride=1 << 41, head_stride=512, row_stride=32), 2, "too large"),
    (dict(page_stride=1 << 35, head_stride=512, row_stride=32, num_pages=1 << 20), 2, "2^48"),
    (dict(page_stride=1 << 36, head_stride=512, row_stride=32), 2, "too large"),
    (dict(scale_page_stride=1 << 33, scale_head_stride=32, scale_row_stride=2), 2, "too large"),
    (dict(scale_page_stride=64), 1, "scales"),
    (dict(scale_page_stride=64, scale_head_stride=31, scale_row_stride=2), 1, "multiple of 2"),
    (dict(scale_page_stride=64, scale_head_stride=30, scale_row_stride=2), 1, "overlap"),
    (dict(key_out_stride=100), 1, "key_out_stride"),
    (dict(value_out_stride=132), 1, "value_out_stride 132"),
    (dict(workspace=None), 4, "workspace is NULL"),
    (dict(workspace_bytes=255), 4, "workspace_bytes"),
    (dict(key_pages=None), 1, "key_pages"),
    (dict(value_pages=16 * MB * 6 + 8), 1, "value_pages is not 16-byte"),
    (dict(key_scales=None), 1, "key_scales is NULL"),
    (dict(value_scales=16 * MB * 11 + 2), 1, "value_scales is not 4-byte"),
    (dict(query_start=None), 1, "query_start"),
    (dict(page_table=16 * MB + 2), 1, "page_table"),
    (dict(cos_cache=1 << 41), 1, "go together"),
])
def test_refusals(lib, over, status, msg):
    for fn in CALLS:
        assert getattr(lib, fn)(_args(lib, **over), 0) == status, fn
        assert msg in lib.gqaw_last_error(), lib.gqaw_last_error()


@pytest.mark.parametrize("over,fns,msg", [
    (dict(query=None), ("attend", "step"), "query is NULL"),
    (dict(output=16 * MB + 8), ("attend", "step"), "output is not 16-byte"),
    (dict(key=None), ("append", "step"), "key is NULL"),
    (dict(value=4), ("append", "step"), "value is not 16-byte"),
    (dict(key_out=None, value_out=None), ("read",), "key_out and value_out are NULL"),
    (dict(value_out=16 * MB + 8), ("read",), "not 16-byte"),
    (dict(value_out=16 * MB * 12), ("read",), "key_out overlaps value_out"),
    (dict(value_out=16 * MB * 12 + 128, key_out_stride=512, value_out_stride=512), ("read",), "key_out overlaps value_out"),
    (dict(key_out=16 * MB * 10), ("read",), "key_scales overlaps key_out"),
    (dict(output=16 * MB * 6), ("attend", "step"), "value_pages overlaps output"),
    (dict(output=16 * MB), ("attend", "step"), "output overlaps query"),
    (dict(key=16 * MB * 5), ("append", "step"), "key_pages overlaps key"),
    (dict(value_pages=16 * MB * 5), ("append", "step"), "key_pages overlaps value_pages"),
    (dict(value_scales=16 * MB * 5 + 512), ("append", "step"), "key_pages overlaps value_scales"),
    (dict(query=1 << 40), ("attend", "step"), "workspace overlaps query"),
    (dict(cos_cache=(1 << 41) + 1, sin_cache=1 << 42, rotary_cache_len=9), ("append", "step"), "cos_cache"),
])
def test_refusals_of_one_call(lib, over, fns, msg):
    for fn in fns:
        assert getattr(lib, "gqaw_paged_i4_" + fn)(_args(lib, **over), 0) == 1, fn
        assert msg in lib.gqaw_last_error(), lib.gqaw_last_error()


def _reaches_device(lib, fn, **over):
    """A call that no check of the host refuses goes on to look at its workspace, which here is no device's."""
    st = getattr(lib, fn)(_args(lib, **over), 0)
    return st != lib.GQAW_OK and "overlaps" not in lib.gqaw_last_error() and (
        st == lib.GQAW_ECUDA or "device" in lib.gqaw_last_error())


def test_woven_caches_pass(lib):
    """All four parts of a page in one block of 4096 + ... bytes, and keys beside values in a row."""
    base = 16 * MB * 5
    block = dict(page_stride=8192, head_stride=512, row_stride=32, scale_page_stride=4096, scale_head_stride=32, scale_row_stride=2,
                 key_pages=base, value_pages=base + 1024, key_scales=base + 2048, value_scales=base + 2176)
    for fn in CALLS:
        assert _reaches_device(lib, fn, **block), lib.gqaw_last_error()
    row = dict(page_stride=4096, head_stride=2048, row_stride=128, scale_page_stride=2048, scale_head_stride=1024, scale_row_stride=64,
               key_pages=base, value_pages=base + 32, key_scales=base + 64, value_scales=base + 68)
    for fn in CALLS:
        assert _reaches_device(lib, fn, **row), lib.gqaw_last_error()
    bad = dict(row, value_scales=base + 66)
    assert lib.gqaw_paged_i4_append(_args(lib, **bad), 0) == 1


def test_nothing_to_do_needs_no_pointers(lib):
    before = lib.gqaw_launch_count()
    for over in (dict(batch_size=0), dict(total_new_tokens=0, max_new_tokens=0), dict(max_new_tokens=0)):
        x = _args(lib, **over)
        for n in ("query", "key", "value", "output", "key_pages", "value_pages", "page_table", "query_start", "seqlens_k", "workspace"):
            setattr(x.paged, n, None)
        for n in ("key_scales", "value_scales", "key_out", "value_out"):
            setattr(x, n, None)
        for fn in CALLS:
            assert getattr(lib, fn)(x, 0) == lib.GQAW_OK
    assert lib.gqaw_launch_count() == before


def test_struct_and_workspace(lib):
    assert lib.load().gqaw_paged_i4_args_size() == ctypes.sizeof(lib.gqaw_paged_i4_args)
    n = lib.gqaw_paged_i4_workspace_bytes(_args(lib, query=None, workspace=None))
    assert n > 4096 and n % 256 == 0
    assert lib.gqaw_paged_i4_workspace_bytes(_args(lib, head_size=16)) == 0
    for fn in ("gqaw_paged_i4_attend", "gqaw_paged_i4_step"):
        assert getattr(lib, fn)(_args(lib, workspace_bytes=n - 256), 0) == lib.GQAW_EWORKSPACE


def test_binding_checks_shapes(lib):
    D, Nq, Nkv, page = 64, 4, 2, 16
    t = dict(query=torch.zeros(5, Nq * D), key=torch.zeros(5, Nkv * D), value=torch.zeros(5, Nkv, D),
             key_codes=torch.zeros(7, Nkv, page, D // 2, dtype=torch.uint8), value_codes=torch.zeros(7, Nkv, page, D // 2, dtype=torch.uint8),
             key_scales=torch.zeros(7, Nkv, page, 2, dtype=torch.bfloat16), value_scales=torch.zeros(7, Nkv, page, 2, dtype=torch.bfloat16),
             page_table=torch.zeros(3, 4, dtype=torch.int32), query_start=torch.zeros(4, dtype=torch.int32),
             seqlens_k=torch.zeros(3, dtype=torch.int32), max_new_tokens=2, max_sequence_length=64, num_heads=Nq,
             kv_num_heads=Nkv, output=torch.zeros(5, Nq * D), key_out=torch.zeros(5, Nkv * D), value_out=torch.zeros(5, Nkv, D))
    x = lib.make_paged_i4_args(**t)
    a = x.paged
    assert (a.head_size, a.page_size, a.num_pages, a.page_table_width, a.dtype) == (D, page, 7, 4, lib.GQAW_F32)
    assert (a.page_stride, a.head_stride, a.row_stride) == (Nkv * page * 32, page * 32, 32)
    assert (x.scale_page_stride, x.scale_head_stride, x.scale_row_stride) == (Nkv * page * 2, page * 2, 2)
    u8, b16 = torch.uint8, torch.bfloat16
    hir = dict(t, key_codes=torch.zeros(7, page, Nkv, 32, dtype=u8), value_codes=torch.zeros(7, page, Nkv, 32, dtype=u8),
               key_scales=torch.zeros(7, page, Nkv, 2, dtype=b16), value_scales=torch.zeros(7, page, Nkv, 2, dtype=b16))
    x = lib.make_paged_i4_args(**hir, heads_inside_rows=True)
    assert (x.paged.row_stride, x.paged.head_stride, x.scale_row_stride, x.scale_head_stride) == (Nkv * 32, 32, Nkv * 2, 2)
    only = dict(t, query=None, key=None, value=None, output=None, key_out=None, value_out=None)
    for bad in (dict(key_codes=t["key_codes"].to(torch.int8), value_codes=t["key_codes"].to(torch.int8)),
                dict(key_scales=t["key_scales"].float(), value_scales=t["key_scales"].float()),
                dict(key_scales=torch.zeros(7, Nkv, page, 4, dtype=b16), value_scales=torch.zeros(7, Nkv, page, 4, dtype=b16)),
                dict(value_codes=torch.zeros(8, Nkv, page, 32, dtype=u8)), dict(kv_num_heads=4), dict(key_out=torch.zeros(4, Nkv * D)),
                dict(value_out=torch.zeros(5, Nkv * D, dtype=b16)), dict(query=torch.zeros(5, Nq * D, dtype=b16)),
                dict(key_scales=torch.zeros(1, 1, 1, 2, dtype=b16).expand(7, Nkv, page, 2), value_scales=torch.zeros(1, 1, 1, 2, dtype=b16).expand(7, Nkv, page, 2)),
                dict(dtype=torch.float16), dict(workspace=torch.zeros(9, dtype=u8, device="meta")), only):
        with pytest.raises((ValueError, TypeError)):
            lib.make_paged_i4_args(**dict(t, **bad))


def test_codes_times_scales_are_bf16_numbers():
    """A scale of five significant bits times any code is exact in bf16, whatever its exponent above bf16's smallest."""
    for e in (-120, -7, 0, 3, 100):
        s = torch.tensor([(16 + m) * 2.0 ** (e - 4) for m in range(16)], dtype=torch.float64)
        v = (torch.arange(16, dtype=torch.float64) - 8)[:, None] * s
        assert torch.equal(v.to(torch.bfloat16).double(), v)


def test_quantize_definition():
    """The plain form of the codes against the formula in 64 bits: the nearest code, a scale in [top / 7, 17 / 16 top / 7]."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((500, 128)) * 10.0 ** rng.integers(-5, 5, (500, 1))).astype(np.float32)
    codes, scales = i4.quantize(x)
    top = np.abs(x.astype(np.float64)).reshape(500, 4, 32).max(-1)
    s = scales.astype(np.float64)
    assert (s >= top / 7 * (1 - 2.0 ** -24)).all() and (s <= top / 7 * 17 / 16 * (1 + 2.0 ** -23)).all()
    mant = np.frexp(s)[0] * 32
    assert (mant == np.round(mant)).all()
    held = i4.values(torch.from_numpy(codes), torch.from_numpy(scales)).numpy()
    assert (np.abs(held - x).reshape(500, 4, 32) <= s[..., None] * (0.5 + 7 * 2.0 ** -23)).all()
