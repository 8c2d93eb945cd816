"""Test helper: a ragged paged batch, its calls through the C ABI and the comparison."""
from __future__ import annotations

import math

import torch

import paged_reference as ref
from sliding_window_gqa_02_gb300 import gqaw

NAN = float("nan")


class Batch:
    """lens: (S, T) per sequence.  Unowned pages and the rows past a sequence's length hold
    NaN; table entries that nobody needs hold -1."""

    def __init__(self, lens, Nq, Nkv, D, page, dtype, seed=0, heads_inside_rows=False, extra_rows=0, lead_rows=0,
                 window=0, softcap=0.0, sink=False, scale=0.0, norm=False, rotary=0, interleaved=False,
                 filled=True, fused=False, spare_pages=2, smooth=False, position_ids=False):
        dev = torch.device("cuda:0")
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Nq, self.Nkv, self.D, self.page, self.dtype = lens, Nq, Nkv, D, page, dtype
        self.window, self.softcap, self.interleaved, self.hir = window, softcap, interleaved, heads_inside_rows
        self.scale, self.smooth = scale, smooth
        need = [(t + page - 1) // page for _, t in lens]
        pages = sum(need) + spare_pages
        perm = torch.randperm(pages, generator=g)
        width = max([1] + need)
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for i, k in enumerate(need):
            table[i, :k] = perm[at:at + k].to(torch.int32)
            at += k
        n = sum(s for s, _ in lens)
        N = lead_rows + n + extra_rows
        starts = [lead_rows]
        for s, _ in lens:
            starts.append(starts[-1] + s)

        def rnd(*shape):
            return torch.randn(*shape, generator=g).to(dtype)

        if fused:  # one (N, (Nq + 2 Nkv) D) tensor, as a projection leaves it
            qkv = rnd(N, (Nq + 2 * Nkv) * D).to(dev)
            self.q, self.k, self.v = qkv.split([Nq * D, Nkv * D, Nkv * D], 1)
        else:
            self.q, self.k, self.v = (rnd(N, h * D).to(dev) for h in (Nq, Nkv, Nkv))
        shape = (pages, page, Nkv, D) if heads_inside_rows else (pages, Nkv, page, D)
        kp, vp = torch.full(shape, NAN, dtype=dtype), torch.full(shape, NAN, dtype=dtype)
        kr, vr = (x if heads_inside_rows else x.transpose(1, 2) for x in (kp, vp))  # (pages, rows, heads, D)
        for i, (s, t) in enumerate(lens):
            j = torch.arange(t if filled else t - s)
            if len(j):
                at = (table[i].long()[j // page], j % page)
                kr[at], vr[at] = rnd(len(j), Nkv, D), rnd(len(j), Nkv, D)
        if window:  # pages that have left every window are not owned any more
            for i, (s, t) in enumerate(lens):
                for c in range(max(0, t - s - window + 1) // page):
                    table[i, c] = -7
        self.kp, self.vp, self.table = kp.to(dev), vp.to(dev), table.to(dev)
        self.starts = torch.tensor(starts, dtype=torch.int32, device=dev)
        self.seqlens = torch.tensor([t - 1 for _, t in lens], dtype=torch.int32, device=dev)
        self.out = torch.full((N, Nq * D), 7.0, dtype=dtype, device=dev)
        self.sink = (torch.randn(Nq, generator=g) * 2).to(dev) if sink else None
        self.qw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype).to(dev) if norm else None
        self.kw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype).to(dev) if norm else None
        self.max_new = max([0] + [s for s, _ in lens])
        self.max_len = max([0] + [t for _, t in lens])
        self.cos = self.sin = self.ids = None
        if rotary:
            rows = self.max_len + 50
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
        kw = dict(local_window_size=self.window, softcap=self.softcap, scale=self.scale, head_sink=self.sink,
                  smooth_softmax=self.smooth, query_weight=self.qw, key_weight=self.kw, norm_eps=1e-5,
                  cos_cache=self.cos, sin_cache=self.sin, position_ids=self.ids, rotary_interleaved=self.interleaved,
                  heads_inside_rows=self.hir)
        kw.update(over)
        make = lambda ws: gqaw.make_paged_args(self.q, self.k, self.v, self.kp, self.vp, self.table, self.starts,
                                               self.seqlens, self.max_new, self.max_len, self.Nq, self.Nkv, self.out,
                                               workspace=ws, **kw)
        if self.ws is None:
            self.ws = gqaw.new_paged_workspace(make(None), self.q.device, torch.cuda.current_stream().cuda_stream)
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

    def expected_query(self):
        """(value, bound) of the normed and turned query rows."""
        return ref.norm_turn(self.q.reshape(-1, self.Nq, self.D), self.qw, 1e-5, self.cos, self.sin, self.table_pos(),
                             self.interleaved)

    def check_output(self, turned=False, skip=(), parts=1):
        """Every output row against the definition over the cache as it is now.  ``turned``: with
        queries that the call norms and turns, kept in ``parts`` numbers of the type: what each
        leaves is within u of it, so two are within u * u."""
        worst = 0.0
        qv = None
        if turned:
            qv, qb = self.expected_query()
        sink = self.sink if self.sink is not None else (torch.zeros(self.Nq, device=self.q.device) if self.smooth else None)
        for i, (s, t) in enumerate(self.lens):
            if s == 0 or i in skip:
                continue
            k = ref.gather(self.kp, self.table[i], t, self.hir)
            v = ref.gather(self.vp, self.table[i], t, self.hir)
            q = (qv if turned else self.q.reshape(-1, self.Nq, self.D).double())[self.rows(i)]
            rounded = ref.u(self.dtype) ** parts + 64 * ref.F32 if turned else 0.0
            if turned:  # the turn's own error, relative to the row (a bound for every element)
                rounded += float((qb[self.rows(i)] / q.abs().amax(-1, keepdim=True).clamp_min(1e-30)).max()) * 4
            want, bound = ref.attend(q, k, v, t - s, self.window, self.scale or 1 / math.sqrt(self.D), self.softcap, sink,
                                     self.dtype, rounded)
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

    def check_untouched(self):
        """Output rows that belong to no sequence keep their bits."""
        keep = torch.ones(self.out.shape[0], dtype=torch.bool)
        for i in range(len(self.lens)):
            keep[self.rows(i)] = False
        assert (self.out[keep.to(self.out.device)] == 7.0).all()

    def check_pages(self, before_k, before_v):
        """Pages after an append: the new rows as the formula gives them (keys within one
        rounding and the arithmetic's error, values bit for bit), all others as before."""
        bits = {2: torch.int16, 4: torch.int32}[self.kp.element_size()]
        want_k, bound = ref.norm_turn(self.k.reshape(-1, self.Nkv, self.D), self.kw, 1e-5, self.cos, self.sin,
                                      self.table_pos(), self.interleaved)
        kp, vp = (x if self.hir else x.transpose(1, 2) for x in (self.kp, self.vp))
        bk, bv = (x if self.hir else x.transpose(1, 2) for x in (before_k, before_v))
        new = torch.zeros(kp.shape[:2], dtype=torch.bool, device=kp.device)
        for i, (s, t) in enumerate(self.lens):
            if s == 0:
                continue
            j = torch.arange(t - s, t, device=kp.device)
            pg, at, rows = self.table[i].long()[j // self.page], j % self.page, self.rows(i)
            have = pg >= 0
            pg, at = pg[have], at[have]
            new[pg, at] = True
            w, got = want_k[rows][have], kp[pg, at].double()
            tol = bound[rows][have] + ref.u(self.dtype) * (w.abs() + bound[rows][have])
            assert ((got - w).abs() <= tol).all(), (i, float(((got - w).abs() - tol).max()))
            if self.kw is None and self.cos is None:
                assert torch.equal(kp[pg, at].view(bits), self.k[rows].reshape(s, self.Nkv, self.D)[have].view(bits))
            assert torch.equal(vp[pg, at].view(bits), self.v[rows].reshape(s, self.Nkv, self.D)[have].view(bits))
        old = ~new
        assert torch.equal(kp[old].view(bits), bk[old].view(bits)) and torch.equal(vp[old].view(bits), bv[old].view(bits))
