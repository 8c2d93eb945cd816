"""Plain 64-bit forms of the paged operators and the per-head norms, for the tests, with the
error that a kernel may make derived beside each value.

Every function works on torch tensors and returns float64.  ``u(dtype)`` is half a step of the
type relative to the value: what one rounding may be off.
"""
from __future__ import annotations

import math

import torch

F32 = 2.0 ** -24  # half a step of the arithmetic


def u(dtype):
    return torch.finfo(dtype).eps / 2


def norm_turn(x, weight, eps, cos, sin, pos, interleaved):
    """x (N, H, D) -> (value, bound on |fp32 result before its rounding - value|).

    The sum of D squares, the mean, the root and its reciprocal, and two products per element
    are at most (log2(D) + 8 + 8) roundings of the norm's factor and the element together (the
    sum is a tree over lanes of 8-term chains, and its error counts half: a square root
    follows); the turn adds two roundings of each product.  32 roundings cover both.
    """
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    size = y.abs()
    if cos is not None:
        rd = 2 * cos.shape[1]
        c, s = cos.double()[pos][:, None, :], sin.double()[pos][:, None, :]
        out, size = y.clone(), size.clone()
        if interleaved:
            ia, ib = torch.arange(0, rd, 2), torch.arange(1, rd, 2)
        else:
            ia, ib = torch.arange(0, rd // 2), torch.arange(rd // 2, rd)
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = (a * c).abs() + (b * s).abs()
        size[..., ib] = (b * c).abs() + (a * s).abs()
        y = out
    return y, 32 * F32 * size


def gather(pages, table_row, length, heads_inside_rows=False):
    """Rows [0, length) of one sequence: (length, heads, D) float64; rows of pages that the
    table does not name are zero."""
    p = pages if heads_inside_rows else pages.transpose(1, 2)  # (pages, rows, heads, D)
    ids = table_row[:(length + p.shape[1] - 1) // p.shape[1]].to(pages.device).long()
    rows = p[ids.clamp(0, p.shape[0] - 1)].double()
    rows = torch.where((ids >= 0)[:, None, None, None], rows, 0.0)
    return rows.reshape(-1, p.shape[2], p.shape[3])[:length]


def attend(q, k, v, first, window, scale, softcap, sink, dtype, q_rounded=0.0):
    """q (S, Nq, D) float64 at positions first ..; k, v (T, Nkv, D) -> (out, bound).

    The bound on |result - out|, rounding of the result included: with a row's weights p,
      - a logit is a sum of D products and a scale (D + 4 roundings of sum |q k| scale), more
        with a rounded query (q_rounded relative to each element); an error dz of every logit
        moves the weights by at most 2 dz relative;
      - a tanh adds 2^-21 of the cap; 2^x, the sums over T keys and their rescalings add
        (T + 64) roundings;
      - a 16-bit kernel rounds each weight for its matrix product: u relative;
      - the result is rounded once.
    Everything but the last is relative to sum p |v|.
    """
    S, Nq, D = q.shape
    T, Nkv, _ = k.shape
    g = Nq // Nkv
    j = torch.arange(T, device=q.device)
    i = first + torch.arange(S, device=q.device)
    seen = j[None, :] <= i[:, None]
    if window:
        seen = seen & (j[None, :] > i[:, None] - window)
    kk, vv = (x.transpose(0, 1)[:, None] for x in (k, v))  # (Nkv, 1, T, D)
    qq = q.reshape(S, Nkv, g, D).permute(1, 2, 0, 3)       # (Nkv, g, S, D)
    z = qq @ kk.transpose(-1, -2) * scale
    size = (qq.abs() @ kk.abs().transpose(-1, -2)) * scale
    size = torch.where(seen, size, 0.0).amax(-1, keepdim=True)
    if softcap:
        z = torch.tanh(z / softcap) * softcap
    z = torch.where(seen, z, -math.inf)
    top = z.amax(-1, keepdim=True)
    if sink is not None:
        sk = sink.double().reshape(Nkv, g, 1, 1)
        top = torch.maximum(top, sk)
    p = torch.exp(z - top)
    den = p.sum(-1, keepdim=True)
    if sink is not None:
        den = den + torch.exp(sk - top)
    p = torch.where(seen, p / den, 0.0)
    # rows of v that a query does not see must not count, whatever they hold
    clean = torch.nan_to_num(vv, nan=0.0, posinf=0.0, neginf=0.0)
    out = p @ clean
    for jj in torch.nonzero(~torch.isfinite(v).all(-1).all(-1)).flatten().tolist():
        odd = torch.where(torch.isfinite(vv[:, :, jj]), 0.0, vv[:, :, jj])  # (Nkv, 1, D)
        for s in torch.nonzero(seen[:, jj]).flatten().tolist():
            out[:, :, s] += torch.where(odd == 0, 0.0, p[:, :, s, jj, None] * odd)
    dz = (D + 4) * F32 * size + q_rounded * size + (2.0 ** -21 * softcap if softcap else 0.0)
    rel = 2 * dz + (T + 64) * F32 + (u(dtype) if dtype == torch.bfloat16 else 0.0)
    bound = rel * (p @ clean.abs()) + u(dtype) * out.abs() * (1 + rel)
    back = lambda x: x.permute(2, 0, 1, 3).reshape(S, Nq, D)
    return back(out), back(bound)
