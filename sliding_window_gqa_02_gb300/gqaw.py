"""ctypes binding of ``libgqaw.so`` (include/gqaw.h), with the same function names.

This module only marshals arguments: every step of the computation runs in the CUDA
kernels of the library.  If the library has not been built the first call raises;
there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libgqaw.so")

GQAW_OK = 0
GQAW_EINVAL = 1
GQAW_EUNSUPPORTED = 2
GQAW_ECUDA = 3
GQAW_EWORKSPACE = 4
GQAW_EDEVICE = 5

GQAW_F32 = 0
GQAW_BF16 = 1

GQAW_I8 = 2
GQAW_E4M3 = 3
GQAW_DEV_BAD_SEQLEN = 1
GQAW_DEV_TIMEOUT = 2
GQAW_DEV_BAD_POSITION = 4
GQAW_DEV_QUERY_RANGE = 8
GQAW_DEV_INTERNAL = 16
GQAW_DEV_BAD_PAGE = 32

STATUS_NAMES = {0: "GQAW_OK", 1: "GQAW_EINVAL", 2: "GQAW_EUNSUPPORTED", 3: "GQAW_ECUDA",
                4: "GQAW_EWORKSPACE", 5: "GQAW_EDEVICE"}

EXPORTED = ["gqaw_resident_len", "gqaw_rollback_exact", "gqaw_workspace_bytes", "gqaw_workspace_init",
            "gqa_windowed_step", "gqaw_attend", "gqaw_update_cache", "gqaw_device_status",
            "gqaw_last_error", "gqaw_launch_count", "gqaw_step_args_size", "gqa_windowed_step_noalloc",
            "gqaw_qk_norm_rotary", "gqaw_paged_workspace_bytes", "gqaw_paged_append", "gqaw_paged_attend",
            "gqaw_paged_step", "gqaw_qk_args_size", "gqaw_paged_args_size",
            "gqaw_paged_i4_workspace_bytes", "gqaw_paged_i4_append", "gqaw_paged_i4_attend", "gqaw_paged_i4_step",
            "gqaw_paged_i4_read", "gqaw_paged_i4_args_size"]

GQAW_I4_GROUP = 32

GQAW_NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024


class gqaw_step_args(ctypes.Structure):
    """Mirror of ``gqaw_step_args`` in include/gqaw.h (same field order and types)."""

    _fields_ = [
        ("batch_size", ctypes.c_int32),
        ("sequence_length", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("kv_num_heads", ctypes.c_int32),
        ("head_size", ctypes.c_int32),
        ("capacity", ctypes.c_int32),
        ("local_window_size", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("softcap", ctypes.c_float),
        ("total_sequence_length", ctypes.c_int32),
        ("split_keys", ctypes.c_int32),
        ("query", ctypes.c_void_p),
        ("key", ctypes.c_void_p),
        ("value", ctypes.c_void_p),
        ("past_key", ctypes.c_void_p),
        ("past_value", ctypes.c_void_p),
        ("present_key", ctypes.c_void_p),
        ("present_value", ctypes.c_void_p),
        ("seqlens_k", ctypes.c_void_p),
        ("attention_bias", ctypes.c_void_p),
        ("bias_stride_b", ctypes.c_int64),
        ("bias_stride_h", ctypes.c_int64),
        ("bias_stride_s", ctypes.c_int64),
        ("output", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("resident_len_out", ctypes.c_void_p),
        ("head_sink", ctypes.c_void_p),
        ("smooth_softmax", ctypes.c_int32),
        ("do_rotary", ctypes.c_int32),
        ("rotary_interleaved", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("rotary_cache_len", ctypes.c_int32),
        ("cos_cache", ctypes.c_void_p),
        ("sin_cache", ctypes.c_void_p),
        ("position_ids", ctypes.c_void_p),
        ("cache_dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
    ]


class gqaw_qk_args(ctypes.Structure):
    """Mirror of ``gqaw_qk_args`` in include/gqaw.h."""

    _fields_ = [
        ("num_tokens", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("kv_num_heads", ctypes.c_int32),
        ("head_size", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("norm_eps", ctypes.c_float),
        ("query", ctypes.c_void_p),
        ("key", ctypes.c_void_p),
        ("query_out", ctypes.c_void_p),
        ("key_out", ctypes.c_void_p),
        ("query_stride", ctypes.c_int64),
        ("key_stride", ctypes.c_int64),
        ("query_out_stride", ctypes.c_int64),
        ("key_out_stride", ctypes.c_int64),
        ("query_weight", ctypes.c_void_p),
        ("key_weight", ctypes.c_void_p),
        ("cos_cache", ctypes.c_void_p),
        ("sin_cache", ctypes.c_void_p),
        ("position_ids", ctypes.c_void_p),
        ("rotary_interleaved", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("rotary_cache_len", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class gqaw_paged_args(ctypes.Structure):
    """Mirror of ``gqaw_paged_args`` in include/gqaw.h."""

    _fields_ = [
        ("batch_size", ctypes.c_int32),
        ("total_new_tokens", ctypes.c_int32),
        ("max_new_tokens", ctypes.c_int32),
        ("max_sequence_length", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("kv_num_heads", ctypes.c_int32),
        ("head_size", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("page_table_width", ctypes.c_int32),
        ("local_window_size", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("softcap", ctypes.c_float),
        ("norm_eps", ctypes.c_float),
        ("smooth_softmax", ctypes.c_int32),
        ("query", ctypes.c_void_p),
        ("key", ctypes.c_void_p),
        ("value", ctypes.c_void_p),
        ("output", ctypes.c_void_p),
        ("query_stride", ctypes.c_int64),
        ("key_stride", ctypes.c_int64),
        ("value_stride", ctypes.c_int64),
        ("output_stride", ctypes.c_int64),
        ("key_pages", ctypes.c_void_p),
        ("value_pages", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
        ("page_table", ctypes.c_void_p),
        ("query_start", ctypes.c_void_p),
        ("seqlens_k", ctypes.c_void_p),
        ("head_sink", ctypes.c_void_p),
        ("query_weight", ctypes.c_void_p),
        ("key_weight", ctypes.c_void_p),
        ("cos_cache", ctypes.c_void_p),
        ("sin_cache", ctypes.c_void_p),
        ("position_ids", ctypes.c_void_p),
        ("rotary_interleaved", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("rotary_cache_len", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class gqaw_paged_i4_args(ctypes.Structure):
    """Mirror of ``gqaw_paged_i4_args`` in include/gqaw.h."""

    _fields_ = [
        ("paged", gqaw_paged_args),
        ("key_scales", ctypes.c_void_p),
        ("value_scales", ctypes.c_void_p),
        ("scale_page_stride", ctypes.c_int64),
        ("scale_head_stride", ctypes.c_int64),
        ("scale_row_stride", ctypes.c_int64),
        ("key_out", ctypes.c_void_p),
        ("value_out", ctypes.c_void_p),
        ("key_out_stride", ctypes.c_int64),
        ("value_out_stride", ctypes.c_int64),
    ]


class GqawError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), message))
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load the library (once).  Raises if it is missing: there is no CPU path."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libgqaw.so is not built (%s); run __graft_entry__.build()" % path)
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(gqaw_step_args)
    lib.gqaw_resident_len.restype = ctypes.c_int64
    lib.gqaw_resident_len.argtypes = [ctypes.c_int64] * 3
    lib.gqaw_rollback_exact.restype = ctypes.c_int
    lib.gqaw_rollback_exact.argtypes = [ctypes.c_int64] * 4
    lib.gqaw_workspace_bytes.restype = ctypes.c_size_t
    lib.gqaw_workspace_bytes.argtypes = [P]
    lib.gqaw_workspace_init.restype = ctypes.c_int
    lib.gqaw_workspace_init.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    for name in ("gqa_windowed_step", "gqaw_attend", "gqaw_update_cache", "gqa_windowed_step_noalloc"):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [P, ctypes.c_void_p]
    lib.gqaw_device_status.restype = ctypes.c_int
    lib.gqaw_device_status.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int,
                                       ctypes.c_void_p]
    lib.gqaw_last_error.restype = ctypes.c_char_p
    lib.gqaw_last_error.argtypes = []
    lib.gqaw_launch_count.restype = ctypes.c_uint64
    lib.gqaw_launch_count.argtypes = []
    lib.gqaw_qk_norm_rotary.restype = ctypes.c_int
    lib.gqaw_qk_norm_rotary.argtypes = [ctypes.POINTER(gqaw_qk_args), ctypes.c_void_p]
    PP = ctypes.POINTER(gqaw_paged_args)
    lib.gqaw_paged_workspace_bytes.restype = ctypes.c_size_t
    lib.gqaw_paged_workspace_bytes.argtypes = [PP]
    for name in ("gqaw_paged_append", "gqaw_paged_attend", "gqaw_paged_step"):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [PP, ctypes.c_void_p]
    PI = ctypes.POINTER(gqaw_paged_i4_args)
    lib.gqaw_paged_i4_workspace_bytes.restype = ctypes.c_size_t
    lib.gqaw_paged_i4_workspace_bytes.argtypes = [PI]
    for name in ("gqaw_paged_i4_append", "gqaw_paged_i4_attend", "gqaw_paged_i4_step", "gqaw_paged_i4_read"):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [PI, ctypes.c_void_p]
    for name, struct in (("gqaw_step_args", gqaw_step_args), ("gqaw_qk_args", gqaw_qk_args),
                         ("gqaw_paged_args", gqaw_paged_args), ("gqaw_paged_i4_args", gqaw_paged_i4_args)):
        size = getattr(lib, name + "_size")
        size.restype = ctypes.c_size_t
        size.argtypes = []
        if size() != ctypes.sizeof(struct):
            raise RuntimeError("%s layout mismatch: library %d bytes, binding %d bytes"
                               % (name, size(), ctypes.sizeof(struct)))
    _lib = lib
    return lib


# ----------------------------------------------------------------- same-name wrappers


def gqaw_resident_len(T: int, C: int, W: int) -> int:
    return int(load().gqaw_resident_len(T, C, W))


def gqaw_rollback_exact(T: int, k: int, C: int, W: int) -> int:
    return int(load().gqaw_rollback_exact(T, k, C, W))


def gqaw_workspace_bytes(args: gqaw_step_args) -> int:
    return int(load().gqaw_workspace_bytes(ctypes.byref(args)))


def gqaw_workspace_init(workspace: int, nbytes: int, stream: int = 0) -> int:
    return int(load().gqaw_workspace_init(workspace, nbytes, stream))


def gqa_windowed_step(args: gqaw_step_args, stream: int = 0) -> int:
    return int(load().gqa_windowed_step(ctypes.byref(args), stream))


def gqa_windowed_step_noalloc(args: gqaw_step_args, stream: int = 0) -> int:
    """The step with its scratch taken from the library's static array (for callers
    that cannot allocate); ``args.workspace`` is ignored."""
    return int(load().gqa_windowed_step_noalloc(ctypes.byref(args), stream))


def gqaw_attend(args: gqaw_step_args, stream: int = 0) -> int:
    return int(load().gqaw_attend(ctypes.byref(args), stream))


def gqaw_update_cache(args: gqaw_step_args, stream: int = 0) -> int:
    return int(load().gqaw_update_cache(ctypes.byref(args), stream))


def gqaw_qk_norm_rotary(args: gqaw_qk_args, stream: int = 0) -> int:
    return int(load().gqaw_qk_norm_rotary(ctypes.byref(args), stream))


def gqaw_paged_workspace_bytes(args: gqaw_paged_args) -> int:
    return int(load().gqaw_paged_workspace_bytes(ctypes.byref(args)))


def gqaw_paged_append(args: gqaw_paged_args, stream: int = 0) -> int:
    return int(load().gqaw_paged_append(ctypes.byref(args), stream))


def gqaw_paged_attend(args: gqaw_paged_args, stream: int = 0) -> int:
    return int(load().gqaw_paged_attend(ctypes.byref(args), stream))


def gqaw_paged_step(args: gqaw_paged_args, stream: int = 0) -> int:
    return int(load().gqaw_paged_step(ctypes.byref(args), stream))


def gqaw_paged_i4_workspace_bytes(args: gqaw_paged_i4_args) -> int:
    return int(load().gqaw_paged_i4_workspace_bytes(ctypes.byref(args)))


def gqaw_paged_i4_append(args: gqaw_paged_i4_args, stream: int = 0) -> int:
    return int(load().gqaw_paged_i4_append(ctypes.byref(args), stream))


def gqaw_paged_i4_attend(args: gqaw_paged_i4_args, stream: int = 0) -> int:
    return int(load().gqaw_paged_i4_attend(ctypes.byref(args), stream))


def gqaw_paged_i4_step(args: gqaw_paged_i4_args, stream: int = 0) -> int:
    return int(load().gqaw_paged_i4_step(ctypes.byref(args), stream))


def gqaw_paged_i4_read(args: gqaw_paged_i4_args, stream: int = 0) -> int:
    return int(load().gqaw_paged_i4_read(ctypes.byref(args), stream))


def gqaw_device_status(workspace: int, reset: bool = False, stream: int = 0):
    """Returns (status, flags)."""
    flags = ctypes.c_uint32(0)
    st = int(load().gqaw_device_status(workspace, ctypes.byref(flags), int(bool(reset)), stream))
    return st, int(flags.value)


def gqaw_last_error() -> str:
    return load().gqaw_last_error().decode()


def gqaw_launch_count() -> int:
    return int(load().gqaw_launch_count())


def check(status: int) -> None:
    if status != GQAW_OK:
        raise GqawError(status, gqaw_last_error())


# ----------------------------------------------------------------- torch marshalling


def _ptr(t):
    return None if t is None else int(t.data_ptr())


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.float32:
        return GQAW_F32
    if t.dtype == torch.bfloat16:
        return GQAW_BF16
    raise TypeError("query/key/value must be float32 or bfloat16, got %s" % t.dtype)


def _cache_code(cache, query) -> int:
    """0 when the caches hold the query's type; GQAW_I8 / GQAW_E4M3 for code caches."""
    import torch

    if cache.dtype == query.dtype:
        return 0
    if cache.dtype == torch.int8:
        return GQAW_I8
    if getattr(torch, "float8_e4m3fn", None) is not None and cache.dtype == torch.float8_e4m3fn:
        return GQAW_E4M3
    raise TypeError("caches must hold the query's type, int8 or float8_e4m3fn, got %s" % cache.dtype)


def make_args(query, key, value, past_key, past_value, present_key, present_value, seqlens_k,
              total_sequence_length: int, num_heads: int, kv_num_heads: int, local_window_size: int,
              output, workspace=None, scale: float = 0.0, softcap: float = 0.0, attention_bias=None,
              bias_strides=None, resident_len_out=None, split_keys: int = 0, head_sink=None,
              smooth_softmax: bool = False, cos_cache=None, sin_cache=None, position_ids=None,
              rotary_interleaved: bool = False, k_scale=None, v_scale=None) -> gqaw_step_args:
    """Fill a ``gqaw_step_args`` from CUDA tensors (shapes as in include/gqaw.h).

    ``attention_bias``: fp32 tensor whose last dimension is contiguous; its (b, h, s)
    strides are taken from the tensor (a size-1 dimension broadcasts with stride 0)
    unless ``bias_strides`` gives them in elements.  ``workspace``: a uint8 CUDA
    tensor, or None when only the size is wanted.  ``head_sink``: None or a contiguous
    fp32 (num_heads,) CUDA tensor of sink logits; ``smooth_softmax``: a sink of 0.
    ``cos_cache``/``sin_cache``: contiguous (max_pos, rd/2) CUDA tensors of the step's
    dtype; giving them turns on the rotary embedding (rd = twice their width);
    ``position_ids``: None or a contiguous int64 (B, S) CUDA tensor.  Caches of dtype
    int8 or float8_e4m3fn make a quantized cache; ``k_scale`` / ``v_scale`` are then
    one-element float32 CUDA tensors.
    """
    B, Nkv, C, D = past_key.shape
    S = query.shape[1]
    a = gqaw_step_args()
    a.batch_size, a.sequence_length = int(B), int(S)
    a.num_heads, a.kv_num_heads, a.head_size = int(num_heads), int(kv_num_heads), int(D)
    a.capacity, a.local_window_size = int(C), int(local_window_size)
    a.dtype = _dtype_code(query)
    a.cache_dtype = _cache_code(past_key, query)
    if a.cache_dtype:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is None or str(t.dtype) != "torch.float32" or t.numel() != 1:
                raise ValueError("%s: a one-element float32 tensor is needed for a quantized cache" % name)
        a.k_scale, a.v_scale = _ptr(k_scale), _ptr(v_scale)
    a.scale, a.softcap = float(scale), float(softcap)
    a.total_sequence_length, a.split_keys = int(total_sequence_length), int(split_keys)
    a.query, a.key, a.value = _ptr(query), _ptr(key), _ptr(value)
    a.past_key, a.past_value = _ptr(past_key), _ptr(past_value)
    a.present_key, a.present_value = _ptr(present_key), _ptr(present_value)
    a.seqlens_k = _ptr(seqlens_k)
    if attention_bias is not None:
        if attention_bias.stride(-1) != 1:
            raise ValueError("attention_bias: last dimension must be contiguous")
        if bias_strides is None:
            bb, bh, bs, _ = attention_bias.shape
            st = attention_bias.stride()
            bias_strides = (0 if bb == 1 else st[0], 0 if bh == 1 else st[1], 0 if bs == 1 else st[2])
        a.attention_bias = _ptr(attention_bias)
        a.bias_stride_b, a.bias_stride_h, a.bias_stride_s = (int(x) for x in bias_strides)
    a.output = _ptr(output)
    if workspace is not None:
        a.workspace, a.workspace_bytes = _ptr(workspace), int(workspace.numel() * workspace.element_size())
    a.resident_len_out = _ptr(resident_len_out)
    if head_sink is not None:
        if str(head_sink.dtype) != "torch.float32" or tuple(head_sink.shape) != (int(num_heads),) \
                or not head_sink.is_contiguous():
            raise ValueError("head_sink: contiguous float32 tensor of shape (num_heads,)")
        a.head_sink = _ptr(head_sink)
    a.smooth_softmax = int(bool(smooth_softmax))
    if cos_cache is not None:
        if sin_cache is None or tuple(sin_cache.shape) != tuple(cos_cache.shape) or cos_cache.dim() != 2 \
                or not (cos_cache.is_contiguous() and sin_cache.is_contiguous()) \
                or cos_cache.dtype != query.dtype or sin_cache.dtype != query.dtype:
            raise ValueError("cos_cache/sin_cache: equal contiguous (max_pos, rd/2) tensors of the query's dtype")
        a.do_rotary, a.rotary_interleaved = 1, int(bool(rotary_interleaved))
        a.rotary_dim, a.rotary_cache_len = 2 * int(cos_cache.shape[1]), int(cos_cache.shape[0])
        a.cos_cache, a.sin_cache = _ptr(cos_cache), _ptr(sin_cache)
        if position_ids is not None:
            if str(position_ids.dtype) != "torch.int64" or tuple(position_ids.shape) != (int(B), int(S)) \
                    or not position_ids.is_contiguous():
                raise ValueError("position_ids: contiguous int64 tensor of shape (B, S)")
            a.position_ids = _ptr(position_ids)
    return a


def new_workspace(args: gqaw_step_args, device, stream: int = 0):
    """Allocate (torch) and zero-initialise a workspace large enough for ``args``."""
    return _new_workspace(gqaw_workspace_bytes(args), device, stream)


def _new_workspace(n: int, device, stream: int):
    import torch

    if n == 0:
        check(GQAW_EINVAL)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    check(gqaw_workspace_init(int(ws.data_ptr()), n, stream))
    return ws


def _rows(name, t, heads: int, head_size: int, like=None):
    """(pointer, element stride between tokens) of (N, heads * D) or (N, heads, D) rows."""
    if t is None:
        return None, 0
    if t.dim() not in (2, 3) or t[0:1].numel() != (heads * head_size if t.shape[0] else 0) or \
            (t.dim() == 3 and tuple(t.shape[1:]) != (heads, head_size)):
        raise ValueError("%s: shape (N, %d) or (N, %d, %d) is needed, got %s"
                         % (name, heads * head_size, heads, head_size, tuple(t.shape)))
    if heads and t.shape[0] and (t.stride(-1) != 1 or (t.dim() == 3 and heads > 1 and t.stride(1) != head_size)):
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    if t.shape[0] > 1 and t.stride(0) < heads * head_size:  # 0 (an expanded tensor) would mean contiguous rows
        raise ValueError("%s: tokens must not overlap" % name)
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError("%s: must have the dtype and device of the other tensors" % name)
    return _ptr(t), int(t.stride(0)) if t.shape[0] > 1 else 0


def _vector(name, t, n: int, like):
    if t is None:
        return None
    if t.dtype != like.dtype or tuple(t.shape) != (n,) or not t.is_contiguous() or t.device != like.device:
        raise ValueError("%s: contiguous (%d,) tensor of the rows' dtype and device" % (name, n))
    return _ptr(t)


def _index(name, t, dtype: str, shape, like):
    if t is None:
        return None
    if str(t.dtype) != "torch." + dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() \
            or t.device != like.device:
        raise ValueError("%s: contiguous %s tensor of shape %s on the rows' device" % (name, dtype, tuple(shape)))
    return _ptr(t)


def _tables(a, cos_cache, sin_cache, interleaved, like):
    if (cos_cache is None) != (sin_cache is None):
        raise ValueError("cos_cache and sin_cache go together")
    if cos_cache is None:
        return
    for t in (cos_cache, sin_cache):
        # an empty tensor has no address, which would mean no rotation
        if t.dim() != 2 or t.numel() == 0 or tuple(t.shape) != tuple(cos_cache.shape) or not t.is_contiguous() \
                or t.dtype != like.dtype or t.device != like.device:
            raise ValueError("cos_cache/sin_cache: equal contiguous (max_pos, rd/2) tensors of the rows' dtype and device")
    a.cos_cache, a.sin_cache = _ptr(cos_cache), _ptr(sin_cache)
    a.rotary_dim, a.rotary_cache_len = 2 * int(cos_cache.shape[1]), int(cos_cache.shape[0])
    a.rotary_interleaved = int(bool(interleaved))


def _workspace(a, t, like):
    if t is None:
        return
    if t.device != like.device or not t.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on the rows' device")
    a.workspace, a.workspace_bytes = _ptr(t), int(t.numel() * t.element_size())


def make_qk_args(query, key, query_out, key_out, num_heads: int, kv_num_heads: int, head_size: int,
                 query_weight=None, key_weight=None, norm_eps: float = 1e-6, cos_cache=None, sin_cache=None,
                 position_ids=None, rotary_interleaved: bool = False, workspace=None) -> gqaw_qk_args:
    """Fill a ``gqaw_qk_args`` from CUDA tensors.

    ``query``/``query_out``: (N, num_heads * head_size) or (N, num_heads, head_size), the heads
    of a token contiguous, any stride between tokens; ``key``/``key_out`` likewise with
    ``kv_num_heads``.  Either pair may be None (with a head count of 0).  An output may be its
    input.  ``workspace``: a uint8 tensor of at least 256 bytes, needed with a rotation.
    """
    like = query if query is not None else key
    if like is None:
        raise ValueError("query or key is needed")
    a = gqaw_qk_args()
    tokens = {int(t.shape[0]) for t in (query, key, query_out, key_out) if t is not None}
    if len(tokens) != 1:
        raise ValueError("query, key and the outputs must have the same number of tokens")
    a.num_tokens = tokens.pop()
    a.num_heads, a.kv_num_heads, a.head_size = int(num_heads), int(kv_num_heads), int(head_size)
    a.dtype, a.norm_eps = _dtype_code(like), float(norm_eps)
    a.query, a.query_stride = _rows("query", query, num_heads, head_size, like)
    a.query_out, a.query_out_stride = _rows("query_out", query_out, num_heads, head_size, like)
    a.key, a.key_stride = _rows("key", key, kv_num_heads, head_size, like)
    a.key_out, a.key_out_stride = _rows("key_out", key_out, kv_num_heads, head_size, like)
    a.query_weight = _vector("query_weight", query_weight, head_size, like)
    a.key_weight = _vector("key_weight", key_weight, head_size, like)
    _tables(a, cos_cache, sin_cache, rotary_interleaved, like)
    a.position_ids = _index("position_ids", position_ids, "int64", (a.num_tokens,), like)
    _workspace(a, workspace, like)
    return a


def _page_strides(pages, kv_num_heads: int, heads_inside_rows: bool):
    """(page size, page stride, head stride, row stride) of a 4-dimensional tensor of pages, in its elements."""
    n, d1, d2, D = (int(x) for x in pages.shape)
    heads, page = (d2, d1) if heads_inside_rows else (d1, d2)
    if heads != kv_num_heads:
        raise ValueError("the pages hold %d kv heads, not %d" % (heads, kv_num_heads))
    st = pages.stride()
    # a dimension of one element may have any stride: one that cannot overlap is given instead
    row, head = (int(st[1]), int(st[2])) if heads_inside_rows else (int(st[2]), int(st[1]))
    if page == 1:
        row = head * heads if heads > 1 else D
    if heads == 1:
        head = row * page
    return page, int(st[0]) if n > 1 else max(row * page, head * heads), head, row


def _equal_pages(names: str, k, v):
    if k.dim() != 4 or tuple(k.shape) != tuple(v.shape) or k.dtype != v.dtype or k.device != v.device:
        raise ValueError("%s: equal 4-dimensional tensors" % names)
    if tuple(k.stride()) != tuple(v.stride()) or k.stride(-1) != 1:
        raise ValueError("%s: equal strides, the last dimension contiguous" % names)
    if any(n > 1 and st < k.shape[3] for n, st in zip(k.shape[:3], k.stride()[:3])):
        raise ValueError("%s: rows must not overlap" % names)


def make_paged_args(query, key, value, key_pages, value_pages, page_table, query_start, seqlens_k,
                    max_new_tokens: int, max_sequence_length: int, num_heads: int, kv_num_heads: int, output,
                    workspace=None, local_window_size: int = 0, scale: float = 0.0, softcap: float = 0.0,
                    head_sink=None, smooth_softmax: bool = False, query_weight=None, key_weight=None,
                    norm_eps: float = 1e-6, cos_cache=None, sin_cache=None, position_ids=None,
                    rotary_interleaved: bool = False, heads_inside_rows: bool = False) -> gqaw_paged_args:
    """Fill a ``gqaw_paged_args`` from CUDA tensors.

    ``key_pages``/``value_pages``: (pages, kv heads, page size, D), or with ``heads_inside_rows``
    (pages, page size, kv heads, D); the last dimension contiguous, the others strided alike
    in both.  ``query``/``output``: (N, num_heads * D) or (N, num_heads, D); ``key``/``value``
    likewise with ``kv_num_heads``; None where the call does not use them (an append needs no
    query and output, an attention no key and value).  ``page_table``: (B, width) int32;
    ``query_start``: (B + 1,) int32; ``seqlens_k``: (B,) int32, each sequence's length
    including its new tokens, less one.  ``workspace``: a uint8 tensor, or None when only the
    size is wanted.  The rest as in ``make_args``.
    """
    _equal_pages("key_pages and value_pages", key_pages, value_pages)
    D = int(key_pages.shape[3])
    a = gqaw_paged_args()
    a.page_size, a.page_stride, a.head_stride, a.row_stride = _page_strides(key_pages, kv_num_heads, heads_inside_rows)
    _paged_common(a, key_pages, page_table, query_start, seqlens_k, max_new_tokens, max_sequence_length, num_heads,
                  kv_num_heads, D, local_window_size, scale, softcap, head_sink, smooth_softmax, query_weight, key_weight,
                  norm_eps, cos_cache, sin_cache, position_ids, rotary_interleaved, workspace,
                  dict(query=query, key=key, value=value, output=output))
    a.num_pages = int(key_pages.shape[0])
    a.key_pages, a.value_pages = _ptr(key_pages), _ptr(value_pages)
    return a


def _paged_common(a, like, page_table, query_start, seqlens_k, max_new_tokens, max_sequence_length, num_heads,
                  kv_num_heads, D, local_window_size, scale, softcap, head_sink, smooth_softmax, query_weight, key_weight,
                  norm_eps, cos_cache, sin_cache, position_ids, rotary_interleaved, workspace, rows, more=()):
    """The fields of ``gqaw_paged_args`` that do not depend on how the cache holds its rows.  ``like``:
    the dtype and device of everything outside it; ``more``: further tensors of a row per token."""
    B, width = (int(x) for x in page_table.shape)
    tokens = {int(t.shape[0]) for t in (*rows.values(), *more) if t is not None}
    if len(tokens) != 1:
        raise ValueError("query, key, value and output must have the same number of tokens")
    a.batch_size, a.total_new_tokens = B, tokens.pop()
    a.max_new_tokens, a.max_sequence_length = int(max_new_tokens), int(max_sequence_length)
    a.num_heads, a.kv_num_heads, a.head_size = int(num_heads), int(kv_num_heads), D
    a.page_table_width = width
    a.local_window_size, a.dtype = int(local_window_size), _dtype_code(like)
    a.scale, a.softcap, a.norm_eps = float(scale), float(softcap), float(norm_eps)
    a.smooth_softmax = int(bool(smooth_softmax))
    for name, heads in (("query", num_heads), ("key", kv_num_heads), ("value", kv_num_heads), ("output", num_heads)):
        ptr, stride = _rows(name, rows[name], heads, D, like)
        setattr(a, name, ptr)
        setattr(a, name + "_stride", stride)
    a.page_table = _index("page_table", page_table, "int32", (B, width), like)
    a.query_start = _index("query_start", query_start, "int32", (B + 1,), like)
    a.seqlens_k = _index("seqlens_k", seqlens_k, "int32", (B,), like)
    a.head_sink = _index("head_sink", head_sink, "float32", (int(num_heads),), like)
    a.query_weight = _vector("query_weight", query_weight, D, like)
    a.key_weight = _vector("key_weight", key_weight, D, like)
    _tables(a, cos_cache, sin_cache, rotary_interleaved, like)
    a.position_ids = _index("position_ids", position_ids, "int64", (a.total_new_tokens,), like)
    _workspace(a, workspace, like)


def make_paged_i4_args(query, key, value, key_codes, value_codes, key_scales, value_scales, page_table, query_start,
                       seqlens_k, max_new_tokens: int, max_sequence_length: int, num_heads: int, kv_num_heads: int, output,
                       key_out=None, value_out=None, workspace=None, local_window_size: int = 0, scale: float = 0.0,
                       softcap: float = 0.0, head_sink=None, smooth_softmax: bool = False, query_weight=None,
                       key_weight=None, norm_eps: float = 1e-6, cos_cache=None, sin_cache=None, position_ids=None,
                       rotary_interleaved: bool = False, heads_inside_rows: bool = False, dtype=None) -> gqaw_paged_i4_args:
    """Fill a ``gqaw_paged_i4_args`` from CUDA tensors.

    ``key_codes``/``value_codes``: uint8 (pages, kv heads, page size, D / 2) and
    ``key_scales``/``value_scales``: bfloat16 (pages, kv heads, page size, D / 32), or with
    ``heads_inside_rows`` (pages, page size, kv heads, ...); the last dimension contiguous, the
    others strided alike for keys and values.  ``key_out``/``value_out``: where a read puts its rows,
    (N, kv_num_heads * D) or (N, kv_num_heads, D).  ``dtype``: that of all rows outside the cache
    (by default the first given row tensor's).  The rest as in ``make_paged_args``.
    """
    import torch
    from types import SimpleNamespace

    _equal_pages("key_codes and value_codes", key_codes, value_codes)
    _equal_pages("key_scales and value_scales", key_scales, value_scales)
    D = 2 * int(key_codes.shape[3])
    if key_codes.dtype != torch.uint8 or key_scales.dtype != torch.bfloat16 or key_scales.device != key_codes.device \
            or tuple(key_scales.shape) != (*key_codes.shape[:3], D // GQAW_I4_GROUP):
        raise ValueError("codes: uint8 (..., D / 2) and scales: bfloat16 (..., D / 32) of the same pages and device")
    rows = dict(query=query, key=key, value=value, output=output)
    if dtype is None:
        given = [t for t in (*rows.values(), key_out, value_out) if t is not None]
        if not given:
            raise ValueError("a row tensor or dtype is needed")
        dtype = given[0].dtype
    like = SimpleNamespace(dtype=dtype, device=key_codes.device)
    x = gqaw_paged_i4_args()
    a = x.paged
    a.page_size, a.page_stride, a.head_stride, a.row_stride = _page_strides(key_codes, kv_num_heads, heads_inside_rows)
    _, x.scale_page_stride, x.scale_head_stride, x.scale_row_stride = _page_strides(key_scales, kv_num_heads,
                                                                                    heads_inside_rows)
    _paged_common(a, like, page_table, query_start, seqlens_k, max_new_tokens, max_sequence_length, num_heads,
                  kv_num_heads, D, local_window_size, scale, softcap, head_sink, smooth_softmax, query_weight, key_weight,
                  norm_eps, cos_cache, sin_cache, position_ids, rotary_interleaved, workspace, rows, (key_out, value_out))
    a.num_pages = int(key_codes.shape[0])
    a.key_pages, a.value_pages = _ptr(key_codes), _ptr(value_codes)
    x.key_scales, x.value_scales = _ptr(key_scales), _ptr(value_scales)
    x.key_out, x.key_out_stride = _rows("key_out", key_out, kv_num_heads, D, like)
    x.value_out, x.value_out_stride = _rows("value_out", value_out, kv_num_heads, D, like)
    return x


def new_paged_i4_workspace(args: gqaw_paged_i4_args, device, stream: int = 0):
    """Allocate (torch) and zero-initialise a workspace large enough for any call with ``args``; appends and reads
    alone take one of 256 bytes that ``gqaw_workspace_init`` has zeroed."""
    return _new_workspace(gqaw_paged_i4_workspace_bytes(args), device, stream)


def new_paged_workspace(args: gqaw_paged_args, device, stream: int = 0):
    """Allocate (torch) and zero-initialise a workspace large enough for ``args``."""
    return _new_workspace(gqaw_paged_workspace_bytes(args), device, stream)
