"""Test helper: a ragged batch over a 4-bit paged cache, its calls through the C ABI and the comparison."""
from __future__ import annotations

import math

import numpy as np
import torch

import i4_reference as i4
import paged_reference as ref
from sliding_window_gqa_02_gb300 import gqaw

NAN = float("nan")


class Batch:
    """lens: (S, T) per sequence.  Rows that no sequence holds have scales that are not numbers and any
    codes; table entries that nobody needs hold -1.  ``woven``: all four parts of a page in one buffer."""

    def __init__(self, lens, Nq, Nkv, D, page, dtype, seed=0, heads_inside_rows=False, extra_rows=0, lead_rows=0,
                 window=0, softcap=0.0, sink=False, scale=0.0, norm=False, rotary=0, interleaved=False, smooth=False,
                 position_ids=False, fused=False, spare_pages=2, woven=False, odd_scales=False, filled=True, max_len=0):
        dev = torch.device("cuda:0")
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Nq, self.Nkv, self.D, self.page, self.dtype = lens, Nq, Nkv, D, page, dtype
        self.window, self.softcap, self.interleaved, self.hir = window, softcap, interleaved, heads_inside_rows
        self.scale, self.smooth, self.odd_scales = scale, smooth, odd_scales
        need = [(t + page - 1) // page for _, t in lens]
        pages = sum(need) + spare_pages
        perm = torch.randperm(pages, generator=g)
        width = max([1, -(-max_len // page)] + need)
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for i, k in enumerate(need):
            table[i, :k] = perm[at:at + k].to(torch.int32)
            at += k
        starts = [lead_rows]
        for s, _ in lens:
            starts.append(starts[-1] + s)
        N = starts[-1] + extra_rows

        def rnd(*shape):
            return torch.randn(*shape, generator=g).to(dtype)

        if fused:
            qkv = rnd(N, (Nq + 2 * Nkv) * D).to(dev)
            self.q, self.k, self.v = qkv.split([Nq * D, Nkv * D, Nkv * D], 1)
        else:
            self.q, self.k, self.v = (rnd(N, h * D).to(dev) for h in (Nq, Nkv, Nkv))
        order = (pages, page, Nkv) if heads_inside_rows else (pages, Nkv, page)
        cd, sd = D // 2, D // i4.GROUP
        parts = []
        if woven:  # a page: key codes, value codes, key scales, value scales
            n = page * Nkv
            size = (n * (2 * cd + 4 * sd) + 15) // 16 * 16
            buf = torch.zeros(pages * size, dtype=torch.uint8, device=dev)
            inner = tuple(torch.empty(order[1:] + (1,)).stride()[:2])
            for k, at in enumerate((0, n * cd)):
                parts.append(buf[at:].as_strided(order + (cd,), (size, inner[0] * cd, inner[1] * cd, 1)))
            half = buf.view(torch.bfloat16)
            for k, at in enumerate((n * cd, n * (cd + sd))):
                parts.append(half[at:].as_strided(order + (sd,), (size // 2, inner[0] * sd, inner[1] * sd, 1)))
        else:
            parts = [torch.zeros(order + (cd,), dtype=torch.uint8, device=dev) for _ in "kv"] + \
                    [torch.zeros(order + (sd,), dtype=torch.bfloat16, device=dev) for _ in "kv"]
        self.kc, self.vc, self.ks, self.vs = parts
        for codes, scales in ((self.kc, self.ks), (self.vc, self.vs)):
            codes.copy_(torch.randint(0, 256, codes.shape, generator=g, dtype=torch.uint8))
            sc = torch.full(scales.shape, NAN, dtype=torch.bfloat16)
            sr = sc if heads_inside_rows else sc.transpose(1, 2)
            for i, (s, t) in enumerate(lens):
                j = torch.arange(t if filled else t - s)
                if len(j):
                    x = torch.rand(len(j), Nkv, sd, generator=g) * 0.3 + 0.1
                    if odd_scales:  # any sign, zero, far apart in size
                        x = x * torch.randint(-1, 2, x.shape, generator=g) * 10.0 ** torch.randint(-2, 2, x.shape, generator=g)
                    else:  # as the append writes them
                        x = torch.from_numpy((x.numpy().view(np.int32) & ~0x7FFFF).view(np.float32))
                    sr[table[i].long()[j // page], j % page] = x.to(torch.bfloat16)
            scales.copy_(sc)
        if window:  # pages that have left every window are not owned any more
            for i, (s, t) in enumerate(lens):
                for c in range(max(0, t - s - window + 1) // page):
                    table[i, c] = -7
        self.table = table.to(dev)
        self.starts = torch.tensor(starts, dtype=torch.int32, device=dev)
        self.seqlens = torch.tensor([t - 1 for _, t in lens], dtype=torch.int32, device=dev)
        self.out = torch.full((N, Nq * D), 7.0, dtype=dtype, device=dev)
        self.ko, self.vo = (torch.full((N, Nkv * D), 7.0, dtype=dtype, device=dev) for _ in "kv")
        self.sink = (torch.randn(Nq, generator=g) * 2).to(dev) if sink else None
        self.qw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype).to(dev) if norm else None
        self.kw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype).to(dev) if norm else None
        self.max_new = max([0] + [s for s, _ in lens])
        self.max_len = max([max_len] + [t for _, t in lens])
        self.cos = self.sin = self.ids = None
        if rotary:
            rows = max([0] + [t for _, t in lens]) + 50
            ang = torch.arange(rows, dtype=torch.float64)[:, None] * 100.0 ** (
                -torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
            self.cos, self.sin = (f(ang).to(dtype).to(dev).contiguous() for f in (torch.cos, torch.sin))
            if position_ids:
                self.ids = torch.randint(0, rows, (N,), generator=g).to(dev)
        self.pos = torch.zeros(N, dtype=torch.int64)
        for i, (s, t) in enumerate(lens):
            self.pos[starts[i]:starts[i] + s] = torch.arange(t - s, t)
        self.ws = None

    def args(self, **over):
        kw = dict(key_out=self.ko, value_out=self.vo, local_window_size=self.window, softcap=self.softcap,
                  scale=self.scale, head_sink=self.sink, smooth_softmax=self.smooth, query_weight=self.qw,
                  key_weight=self.kw, norm_eps=1e-5, cos_cache=self.cos, sin_cache=self.sin, position_ids=self.ids,
                  rotary_interleaved=self.interleaved, heads_inside_rows=self.hir)
        kw.update(over)
        make = lambda ws: gqaw.make_paged_i4_args(
            self.q, self.k, self.v, self.kc, self.vc, self.ks, self.vs, self.table, self.starts, self.seqlens,
            self.max_new, self.max_len, self.Nq, self.Nkv, self.out, workspace=ws, **kw)
        if self.ws is None:
            self.ws = gqaw.new_paged_i4_workspace(make(None), self.q.device, torch.cuda.current_stream().cuda_stream)
        return make(self.ws)

    def call(self, fn, flags=0, **over):
        stream = torch.cuda.current_stream().cuda_stream
        gqaw.check(fn(self.args(**over), stream))
        torch.cuda.synchronize()
        st, got = gqaw.gqaw_device_status(int(self.ws.data_ptr()), reset=True, stream=stream)
        assert got == flags, "device status 0x%x" % got

    def rows(self, i):
        a = int(self.starts[i])
        return slice(a, a + self.lens[i][0])

    def table_pos(self):
        return self.pos.to(self.q.device) if self.ids is None else self.ids

    def held(self):
        """(keys, values) of the cache as float64 (pages, rows, heads, D)."""
        return tuple(i4.values(*(x if self.hir else x.transpose(1, 2) for x in p)) for p in ((self.kc, self.ks), (self.vc, self.vs)))

    def check_output(self, turned=False, skip=()):
        """Every output row against the definition over the cache as it is now.

        ``ref.attend``'s bound, with what these kernels round: a query element is taken in one (bf16) or
        two parts of fp16 after a power of two for its row (2^-23 relative to it, or 2^-39 of the row's
        largest for the smallest ones), turned queries of bf16 in two parts (u^2), and each weight, or
        weight times value scale, to fp16 (2^-12; fp32: two parts, 2^-23), or to bf16 with many rows.

        The types end: a weight of a key below fp32's smallest normal number, 2^-126 of the row's largest,
        may count as nothing, and a result below it is rounded to a multiple of bf16's smallest number, 2^-133.
        In fp16 a weight of 1 times the largest scale s of its group (a weight of 1) is at least 2^12 (2^13),
        and what is rounded to a subnormal is off by up to 2^-25: 2^-37 s, times a code of at most 8, where
        the largest value is at least s or there is none: 2^-34 of it a key.

        Scales that the append did not write: with many rows in bf16 every key and value element is
        rounded once to bf16 (u), the keys' share in a logit like a query's, the values' beside the weights'."""
        rounds = self.odd_scales and self.dtype == torch.bfloat16 and self.max_new * (self.Nq // self.Nkv) > 32
        if turned:
            q32 = torch.from_numpy(i4.norm_turn(self.q.reshape(-1, self.Nq, self.D), self.qw, 1e-5, self.cos, self.sin,
                                                self.table_pos(), self.interleaved)).to(self.q.device).double()
        k_all, v_all = self.held()
        sink = self.sink if self.sink is not None else (torch.zeros(self.Nq, device=self.q.device) if self.smooth else None)
        worst = 0.0
        for i, (s, t) in enumerate(self.lens):
            if s == 0 or i in skip:
                continue
            k, v = (ref.gather(x, self.table[i], t, True) for x in (k_all, v_all))
            q = (q32 if turned else self.q.reshape(-1, self.Nq, self.D).double())[self.rows(i)]
            rounded = (ref.u(self.dtype) ** 2 if turned and self.dtype == torch.bfloat16 else 0.0) + 2.0 ** -22
            rounded += ref.u(self.dtype) if rounds else 0.0
            want, bound = ref.attend(q, k, v, t - s, self.window, self.scale or 1 / math.sqrt(self.D), self.softcap, sink,
                                     self.dtype, rounded)
            top = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0).abs().amax()
            bound = bound + (t + 1) * (2.0 ** -126 * (1 + top) + 2.0 ** -34 * top)
            if rounds:
                bound = bound + ref.u(self.dtype) * ref.attend(q, k, v.abs(), t - s, self.window, self.scale or 1 / math.sqrt(self.D),
                                                               self.softcap, sink, self.dtype)[0]
            got = self.out[self.rows(i)].reshape(s, self.Nq, self.D).double()
            bad = ~torch.isfinite(want)
            assert not (torch.isfinite(got) & bad).any(), "finite output where a visible value is not"
            err = torch.where(bad, 0.0, (got - want).abs())
            over = err - bound
            ok = (over <= 0) | bad
            assert ok.all(), "sequence %d: error %.3g, allowed %.3g at %s" % (
                i, float(err.flatten()[over.flatten().argmax()]), float(bound.flatten()[over.flatten().argmax()]),
                torch.nonzero(~ok)[:4].tolist())
            worst = max(worst, float((err / bound.clamp_min(1e-30)).max()))
        return worst

    def untouched(self):
        keep = torch.ones(self.out.shape[0], dtype=torch.bool)
        for i in range(len(self.lens)):
            keep[self.rows(i)] = False
        return keep.to(self.out.device)

    def snapshot(self):
        return [x.clone() for x in (self.kc, self.vc, self.ks, self.vs)]

    def check_pages(self, before):
        """Codes and scales after an append, bit for bit: the new rows as the formula gives them, all others
        as before."""
        y = i4.norm_turn(self.k.reshape(-1, self.Nkv, self.D), self.kw, 1e-5, self.cos, self.sin, self.table_pos(),
                         self.interleaved)
        x = self.v.reshape(-1, self.Nkv, self.D).float().cpu().numpy()
        new = torch.zeros((self.kc.shape[0], self.page), dtype=torch.bool, device=self.kc.device)
        for codes, scales, was, rows in ((self.kc, self.ks, (before[0], before[2]), y), (self.vc, self.vs, (before[1], before[3]), x)):
            want_c, want_s = i4.quantize(rows)
            c, s, c0, s0 = (t if self.hir else t.transpose(1, 2) for t in (codes, scales, *was))
            for i, (n, t) in enumerate(self.lens):
                if n == 0:
                    continue
                j = torch.arange(t - n, t, device=c.device)
                pg, at = self.table[i].long()[j // self.page], j % self.page
                have = pg >= 0
                new[pg[have], at[have]] = True
                got_c, got_s = c[pg[have], at[have]].cpu(), s[pg[have], at[have]].float().cpu()
                r = self.rows(i)
                m = have.cpu()
                assert torch.equal(got_s, torch.from_numpy(want_s[r])[m]) or torch.equal(
                    torch.nan_to_num(got_s, nan=-1.0), torch.nan_to_num(torch.from_numpy(want_s[r])[m], nan=-1.0)), "scales of sequence %d" % i
                assert torch.equal(got_c, torch.from_numpy(want_c[r])[m]), "codes of sequence %d" % i
            old = ~new
            assert torch.equal(c[old], c0[old]) and torch.equal(s[old].view(torch.int16), s0[old].view(torch.int16))

    def check_read(self, keys=True, vals=True):
        for out, held, want in ((self.ko, self.held()[0], keys), (self.vo, self.held()[1], vals)):
            rows = torch.ones(out.shape[0], dtype=torch.bool, device=out.device)
            for i, (s, t) in enumerate(self.lens):
                if s == 0 or not want:
                    continue
                j = torch.arange(t - s, t, device=out.device)
                pg = self.table[i].long()[j // self.page]
                r = torch.arange(int(self.starts[i]), int(self.starts[i]) + s, device=out.device)[pg >= 0]
                rows[r] = False
                x = held[pg[pg >= 0], (j % self.page)[pg >= 0]].flatten(1).to(self.dtype)  # one rounding
                assert torch.equal(out[r].nan_to_num(nan=9.0), x.nan_to_num(nan=9.0)), "rows of sequence %d" % i
            assert (out[rows] == 7.0).all()
