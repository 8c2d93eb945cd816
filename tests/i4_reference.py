"""Plain forms of the 4-bit cache for the tests: what codes stand for (64 bits), the codes of rows
(numpy, every operation in the precision that the operator's definition gives it), and the norm and
turn with their roundings."""
from __future__ import annotations

import numpy as np
import torch

GROUP = 32


def values(codes, scales):
    """uint8 (..., D / 2), bf16 (..., D / 32) -> float64 (..., D)."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double() - 8.0
    return (c.unflatten(-1, (-1, GROUP)) * scales.double()[..., None]).flatten(-2)


def quantize(y):
    """numpy float32 (..., D) -> (codes uint8 (..., D / 2), scales float32 (..., D / 32))."""
    assert y.dtype == np.float32
    g = y.reshape(*y.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        top = np.abs(g).max(-1)  # a NaN stays
        quot = top / np.float32(7)
        scale = ((quot.view(np.int32).astype(np.int64) + 0x7FFFF) & ~0x7FFFF).astype(np.int32).view(np.float32)
        scale = np.where(np.isfinite(top), scale, np.float32("nan")).astype(np.float32)
        c = np.clip(np.rint(g / scale[..., None]), -7, 7)
        c = np.where(scale[..., None] > 0, c, 0).astype(np.int32) + 8
    c = c.reshape(y.shape).astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), scale


def norm_turn(x, weight, eps, cos, sin, pos, interleaved):
    """Torch (N, H, D) -> numpy float32: the factor of the norm in 64 bits and rounded once, every other
    operation rounded to fp32."""
    f = lambda t: t.detach().cpu().float().numpy()
    y = f(x)
    with np.errstate(all="ignore"):
        if weight is not None:
            sq = np.square(y.astype(np.float64)).mean(-1, keepdims=True) + np.float64(np.float32(eps))
            y = (y * (1.0 / np.sqrt(sq)).astype(np.float32)) * f(weight)
        if cos is not None:
            rd = 2 * cos.shape[1]
            at = pos.detach().cpu().numpy()
            c, s = f(cos)[at][:, None, :], f(sin)[at][:, None, :]
            ia, ib = (np.arange(0, rd, 2), np.arange(1, rd, 2)) if interleaved else (np.arange(rd // 2), np.arange(rd // 2, rd))
            out = y.copy()
            a, b = y[..., ia], y[..., ib]
            out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
            y = out
    assert y.dtype == np.float32
    return y
