"""Cases and plain forms of the paged-cache operators.

Four operators: per-head RMS norm of queries and keys with the rotary embedding in the same
pass (``qk``), the append of keys and values to a paged cache with that norm and rotation on
the way (``append``), attention of a ragged batch of new tokens over a paged cache
(``attend``), and the whole step that runs them together (``step``).

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU, ``run`` computes
one pass (the plain form in 32 bits, or the library's calls when ``own`` is true), ``exact``
the same from the definition in 64 bits.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
THETA = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------------------- cases


def _qk(tokens, nq, nkv, d, dtype, rd=0, interleaved=False, max_pos=32768):
    return dict(op="qk", tokens=tokens, nq=nq, nkv=nkv, d=d, dtype=dtype, rd=rd or d, interleaved=interleaved,
                max_pos=max_pos)


def _paged(op, lens, nq, nkv, d, dtype, page, window=0, softcap=0.0, sink=False, rd=0, interleaved=False, norm=True):
    """lens: "S:T" per sequence, S new tokens ending at length T."""
    return dict(op=op, lens=" ".join("%d:%d" % st for st in lens), nq=nq, nkv=nkv, d=d, dtype=dtype, page=page,
                window=window, softcap=softcap, sink=sink, rd=rd or d, interleaved=interleaved, norm=norm)


def _spread(n, lo, hi, seed):
    """n lengths between lo and hi, log-uniform, from a fixed congruential sequence."""
    out, x = [], seed
    for _ in range(n):
        x = (x * 1103515245 + 12345) % (1 << 31)
        out.append(int(round(lo * (hi / lo) ** (x / float(1 << 31)))))
    return out


def listed():
    cases = []

    def add(name, c):
        c["name"] = name
        cases.append(c)

    # a few sequences' new tokens in fp32, interleaved pairs, half the head turned: a small call
    add("qk-small", _qk(61, 64, 8, 64, F32, rd=32, interleaved=True))
    # the tokens of a prefill step (8 chunks of about 512) in bf16
    add("qk-prefill", _qk(4099, 32, 8, 128, BF16))
    # one decode step of 64 sequences: 64 rows into 64 different pages
    add("append-decode", _paged("append", [(1, t) for t in _spread(64, 256, 2048, 1)], 32, 8, 128, BF16, 16))
    # ragged prompt chunks, one sequence without new tokens
    add("append-chunks", _paged("append", [(512, 512), (512, 1813), (131, 700), (0, 400), (512, 2048), (509, 1021),
                                           (1, 1), (512, 1536)], 32, 8, 128, BF16, 64))
    # one token of one short sequence: latency alone
    add("attend-one", _paged("attend", [(1, 131)], 32, 8, 128, BF16, 16))
    # the long-context decode batch: 64 ragged sequences, every key visible
    add("attend-decode", _paged("attend", [(1, t) for t in _spread(64, 4096, 32768, 2)], 32, 8, 128, BF16, 16))
    # speculative verification: 8 drafted tokens for each of 16 sequences, windowed and capped
    add("attend-verify", _paged("attend", [(8, t) for t in _spread(16, 6008, 6072, 3)], 32, 8, 128, BF16, 32,
                                window=4096, softcap=30.0))
    # chunked prefill: 512 tokens of each of 8 long windowed sequences
    add("attend-prefill", _paged("attend", [(512, t) for t in _spread(8, 4608, 32768, 4)], 32, 8, 128, BF16, 64,
                                 window=4096))
    # continuous batching: decoding sequences, two prompt chunks and two idle sequences in one call
    add("attend-mixed", _paged("attend", [(1, t) for t in _spread(20, 128, 8192, 5)] + [(512, 4000), (333, 333), (0, 77),
                                                                                       (0, 0)],
                               64, 8, 64, BF16, 128, sink=True))
    # decode with an fp32 cache
    add("attend-f32", _paged("attend", [(1, 8192), (1, 2047), (1, 513), (1, 5000)], 64, 8, 64, F32, 16))
    # a whole decode step: norm, rotation, append, attention
    add("step-decode", _paged("step", [(1, t) for t in _spread(32, 512, 4096, 6)], 32, 8, 128, BF16, 16))
    # a whole prompt step: a 2048-token prompt from an empty cache, and a short one behind it
    add("step-prompt", _paged("step", [(2048, 2048), (77, 1077)], 32, 8, 128, BF16, 64))
    return cases


_HEADS = [(32, 8), (64, 8), (16, 16), (16, 2), (8, 1), (28, 4), (12, 4), (10, 2), (7, 1), (40, 8)]


def _logint(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["qk", "append", "attend", "attend", "attend", "step"])
    dtype = BF16 if rng.random() < 0.75 else F32
    nq, nkv = rng.choice(_HEADS)
    d = rng.choice([64, 128, 128, 256] if dtype == BF16 else [32, 64, 128])
    rd = rng.choice([d, d, d // 2])
    inter = rng.random() < 0.3
    if op == "qk":
        return _qk(_logint(rng, 1, 4099), nq, nkv, d, dtype, rd, inter)
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["decode", "verify", "chunks", "mixed"])
    n = _logint(rng, 1, 64 if kind == "decode" else 16)
    top = _logint(rng, 64, 16384)
    cap = 262144 if op == "attend" else 49152  # cache tokens in all
    lens = []
    for i in range(n):
        t = _logint(rng, max(1, top // 8), top)
        if kind == "decode":
            s = 1
        elif kind == "verify":
            s = rng.randint(1, 8)
        elif kind == "chunks":
            s = _logint(rng, 1, 1024)
        else:
            s = rng.choice([0, 1, 1, 1, 1, _logint(rng, 1, 512)])
        s = min(max(s, 0 if lens else 1), t)  # the first sequence has a token
        if sum(x[1] for x in lens) + t > cap and lens:
            break
        lens.append((s, t))
    if dtype == F32:  # fewer new tokens: 32-bit products run at a fraction of the 16-bit rate
        lens = [(min(s, 128), t) for s, t in lens]
    window = rng.choice([0, 0, _logint(rng, 16, 4096)])
    softcap = rng.choice([0.0, 0.0, 30.0])
    return _paged(op, lens, nq, nkv, d, dtype, page, window, softcap, rng.random() < 0.3, rd, inter,
                  rng.random() < 0.7)


# ---------------------------------------------------------------------------- inputs


def _lens(case):
    return [tuple(int(v) for v in w.split(":")) for w in case["lens"].split()]


def _tables(rows, rd, dtype, dev):
    """cos and sin of pos * THETA^(-2i/rd), angles in 64 bits, rounded once."""
    inv = THETA ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=dev) / rd)
    ang = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * inv[None, :]
    return torch.cos(ang).to(dtype).contiguous(), torch.sin(ang).to(dtype).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]
    nq, nkv, d = case["nq"], case["nkv"], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    def weight():
        return (1.0 + 0.1 * torch.randn(d, generator=g, device=dev)).to(dt)

    st = {"case": case}
    if case["op"] == "qk":
        n = case["tokens"]
        st["q"], st["k"] = normal(n, nq * d), normal(n, nkv * d)
        st["qw"], st["kw"] = weight(), weight()
        st["cos"], st["sin"] = _tables(case["max_pos"], case["rd"], dt, dev)
        st["pos"] = torch.randint(0, case["max_pos"], (n,), generator=g, device=dev, dtype=torch.int64)
        st["qo"], st["ko"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        if own:
            from sliding_window_gqa_02_gb300 import gqaw

            ws = torch.empty(256, dtype=torch.uint8, device=dev)
            gqaw.check(gqaw.gqaw_workspace_init(ws.data_ptr(), 256, torch.cuda.current_stream().cuda_stream))
            st["ws"] = ws
            st["args"] = gqaw.make_qk_args(
                st["q"], st["k"], st["qo"], st["ko"], nq, nkv, d, query_weight=st["qw"], key_weight=st["kw"],
                norm_eps=EPS, cos_cache=st["cos"], sin_cache=st["sin"], position_ids=st["pos"],
                rotary_interleaved=case["interleaved"], workspace=ws)
        return st

    lens, page = _lens(case), case["page"]
    b = len(lens)
    n = sum(s for s, _ in lens)
    width = max(1, max((t + page - 1) // page for _, t in lens))
    need = [(t + page - 1) // page for _, t in lens]
    pages = sum(need) + 3  # a few pages that nobody owns
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = perm[at:at + k]
        at += k
    starts = [0]
    for s, _ in lens:
        starts.append(starts[-1] + s)
    st["table"] = table
    st["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    st["seqlens"] = torch.tensor([t - 1 for _, t in lens], dtype=torch.int32, device=dev)
    st["q"] = normal(n, nq * d)
    st["k"], st["v"] = normal(n, nkv * d), normal(n, nkv * d)
    st["kp"], st["vp"] = normal(pages, nkv, page, d), normal(pages, nkv, page, d)
    st["out"] = torch.zeros(n, nq * d, dtype=dt, device=dev)
    st["sink"] = torch.randn(nq, generator=g, device=dev) if case["sink"] else None
    turn = case["op"] != "attend"
    st["qw"] = weight() if turn and case["norm"] else None
    st["kw"] = weight() if turn and case["norm"] else None
    max_len = max(t for _, t in lens)
    st["cos"], st["sin"] = _tables(max_len, case["rd"], dt, dev) if turn else (None, None)
    if own:
        from sliding_window_gqa_02_gb300 import gqaw

        def args(ws):
            return gqaw.make_paged_args(
                st["q"], st["k"], st["v"], st["kp"], st["vp"], table, st["starts"], st["seqlens"],
                max(s for s, _ in lens), max_len, nq, nkv, st["out"], workspace=ws,
                local_window_size=case["window"], softcap=case["softcap"], head_sink=st["sink"],
                query_weight=st["qw"], key_weight=st["kw"], norm_eps=EPS, cos_cache=st["cos"], sin_cache=st["sin"],
                rotary_interleaved=case["interleaved"])

        st["ws"] = gqaw.new_paged_workspace(args(None), dev, torch.cuda.current_stream().cuda_stream)
        st["args"] = args(st["ws"])
    return st


# ---------------------------------------------------------------------------- plain forms (32 bits)


def _norm_turn(x, w, cos, sin, pos, rd, interleaved):
    """x (N, H, D) fp32: RMS norm over D times w, then the first rd dimensions turned."""
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    if cos is None:
        return x
    c, s = cos[pos].float()[:, None, :], sin[pos].float()[:, None, :]
    x = x.clone()
    if interleaved:
        a, b = x[..., 0:rd:2].clone(), x[..., 1:rd:2].clone()
        x[..., 0:rd:2], x[..., 1:rd:2] = a * c - b * s, b * c + a * s
    else:
        h = rd // 2
        a, b = x[..., :h].clone(), x[..., h:rd].clone()
        x[..., :h], x[..., h:rd] = a * c - b * s, b * c + a * s
    return x


def _positions(case, dev):
    return torch.cat([torch.arange(t - s, t, device=dev) for s, t in _lens(case)] + [torch.empty(0, device=dev, dtype=torch.int64)])


def _plain_append(st):
    case = st["case"]
    nkv, d, page = case["nkv"], case["d"], case["page"]
    dev = st["k"].device
    pos = _positions(case, dev)
    seq = torch.cat([torch.full((s,), i, device=dev) for i, (s, _) in enumerate(_lens(case))]).long()
    k = _norm_turn(st["k"].view(-1, nkv, d).float(), st["kw"], st["cos"], st["sin"], pos, case["rd"], case["interleaved"])
    p = st["table"][seq, pos // page].long()
    st["kp"][p, :, pos % page] = k.to(st["kp"].dtype)
    st["vp"][p, :, pos % page] = st["v"].view(-1, nkv, d)


def _plain_attend(st, q):
    """q (N, Nq, D) fp32 against the pages; the rows go to st["out"]."""
    case = st["case"]
    nq, nkv, d, page, w = case["nq"], case["nkv"], case["d"], case["page"], case["window"]
    grp = nq // nkv
    n0 = 0
    for i, (s, t) in enumerate(_lens(case)):
        if s == 0:
            continue
        lo = max(0, t - s - w + 1) if w else 0
        p0, p1 = lo // page, (t - 1) // page + 1
        ids = st["table"][i, p0:p1].long()
        k = st["kp"][ids].permute(1, 0, 2, 3).reshape(nkv, -1, d).float()
        v = st["vp"][ids].permute(1, 0, 2, 3).reshape(nkv, -1, d)[:, :t - p0 * page].float()
        k = k[:, :t - p0 * page]
        key = torch.arange(p0 * page, t, device=q.device)
        for r0 in range(0, s, 512):
            r1 = min(s, r0 + 512)
            at = torch.arange(t - s + r0, t - s + r1, device=q.device)
            qq = q[n0 + r0:n0 + r1].view(r1 - r0, nkv, grp, d).permute(1, 2, 0, 3).reshape(nkv, grp * (r1 - r0), d)
            z = torch.matmul(qq, k.transpose(1, 2)).view(nkv, grp, r1 - r0, -1) / math.sqrt(d)
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            hide = key[None, :] > at[:, None]
            if w:
                hide = hide | (key[None, :] <= at[:, None] - w)
            z = z.masked_fill(hide, float("-inf"))
            m = z.max(-1, keepdim=True).values
            if st["sink"] is not None:
                sk = st["sink"].view(nkv, grp, 1, 1)
                m = torch.maximum(m, sk)
            e = torch.exp(z - m)
            den = e.sum(-1, keepdim=True)
            if st["sink"] is not None:
                den = den + torch.exp(sk - m)
            o = torch.matmul((e / den).view(nkv, grp * (r1 - r0), -1), v)
            o = o.view(nkv, grp, r1 - r0, d).permute(2, 0, 1, 3).reshape(r1 - r0, nq * d)
            st["out"][n0 + r0:n0 + r1] = o.to(st["out"].dtype)
        n0 += s


def run(state):
    st, case = state, state["case"]
    if own:
        from sliding_window_gqa_02_gb300 import gqaw

        stream = torch.cuda.current_stream().cuda_stream
        if case["op"] == "qk":
            gqaw.check(gqaw.gqaw_qk_norm_rotary(st["args"], stream))
            return st["qo"], st["ko"]
        if case["op"] == "append":
            gqaw.check(gqaw.gqaw_paged_append(st["args"], stream))
            return st["kp"], st["vp"]
        if case["op"] == "attend":
            gqaw.check(gqaw.gqaw_paged_attend(st["args"], stream))
            return st["out"]
        gqaw.check(gqaw.gqaw_paged_step(st["args"], stream))
        return st["out"], st["kp"], st["vp"]
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    turn = (st["cos"], st["sin"])
    if case["op"] == "qk":
        tail = (st["pos"], case["rd"], case["interleaved"])
        st["qo"].copy_(_norm_turn(st["q"].view(-1, nq, d).float(), st["qw"], *turn, *tail).view(-1, nq * d))
        st["ko"].copy_(_norm_turn(st["k"].view(-1, nkv, d).float(), st["kw"], *turn, *tail).view(-1, nkv * d))
        return st["qo"], st["ko"]
    if case["op"] == "append":
        _plain_append(st)
        return st["kp"], st["vp"]
    q = st["q"].view(-1, nq, d).float()
    if case["op"] == "attend":
        _plain_attend(st, q)
        return st["out"]
    _plain_append(st)
    q = _norm_turn(q, st["qw"], *turn, _positions(case, q.device), case["rd"], case["interleaved"])
    _plain_attend(st, q)
    return st["out"], st["kp"], st["vp"]


# ---------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    es = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "qk":
        n = case["tokens"]
        rows = n * (nq + nkv)
        return {"bytes": rows * d * es * 2 + 2 * d * es + n * (8 + case["rd"] * es), "flops": rows * (4 * d + 3 * case["rd"])}
    lens, w = _lens(case), case["window"]
    n = sum(s for s, _ in lens)
    index = 4 * (2 * len(lens) + 1)
    append = n * nkv * d * es * 4 + n * (4 + case["rd"] * es) + 3 * n * nkv * d
    if case["op"] == "append":
        return {"bytes": append + index, "flops": n * nkv * (4 * d + 3 * case["rd"])}
    rows = pairs = 0
    for s, t in lens:
        if s == 0:
            continue
        lo = max(0, t - s - w + 1) if w else 0
        rows += t - lo
        pairs += sum(min(i + 1, w) if w else i + 1 for i in range(t - s, t))
        index += 4 * ((t - 1) // case["page"] - lo // case["page"] + 1)
    out = {"bytes": rows * nkv * d * es * 2 + 2 * n * nq * d * es + index, "flops": 4 * pairs * nq * d}
    if case["op"] == "step":  # the new rows are read once from the inputs and written once to the pages
        out["bytes"] += n * nkv * d * es * 2 + n * case["rd"] * es
        out["flops"] += n * (nq + nkv) * (4 * d + 3 * case["rd"])
    return out


# ---------------------------------------------------------------------------- the definition (64 bits)


def _exact_rows(x, w, st, pos, heads):
    """Rows of x (N, heads * D), normed and turned, in float64: the turn as a complex product."""
    case = st["case"]
    d, rd = case["d"], case["rd"]
    y = x.double().reshape(x.shape[0], heads, d)
    if w is not None:
        y = y * w.double() / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
    if st["cos"] is None:
        return y
    turn = torch.complex(st["cos"].double(), st["sin"].double())[pos].unsqueeze(1)
    head, rest = y[..., :rd], y[..., rd:]
    if case["interleaved"]:
        z = torch.view_as_complex(head.reshape(x.shape[0], heads, rd // 2, 2).contiguous()) * turn
        head = torch.view_as_real(z).reshape(x.shape[0], heads, rd)
    else:
        z = torch.complex(head[..., :rd // 2].contiguous(), head[..., rd // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, rest], -1)


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    if case["op"] == "qk":
        return (_exact_rows(st["q"], st["qw"], st, st["pos"], nq).reshape(-1, nq * d),
                _exact_rows(st["k"], st["kw"], st, st["pos"], nkv).reshape(-1, nkv * d))
    lens, page = _lens(case), case["page"]
    kp, vp = st["kp"].double(), st["vp"].double()
    held = None  # the keys as the cache holds them: rounded to its type
    table = st["table"].cpu().tolist()
    if case["op"] != "attend":
        held = kp.clone()
        at = 0
        for i, (s, t) in enumerate(lens):
            if s:
                pos = torch.arange(t - s, t, device=kp.device)
                k = _exact_rows(st["k"][at:at + s], st["kw"], st, pos, nkv)
                v = st["v"][at:at + s].double().reshape(s, nkv, d)
                j = t - s
                while j < t:  # page by page
                    n = min(t - j, page - j % page)
                    p, r, a = table[i][j // page], j % page, j - (t - s)
                    kp[p, :, r:r + n] = k[a:a + n].transpose(0, 1)
                    held[p, :, r:r + n] = k[a:a + n].transpose(0, 1).to(st["kp"].dtype).double()
                    vp[p, :, r:r + n] = v[a:a + n].transpose(0, 1)
                    j += n
            at += s
        if case["op"] == "append":
            return kp, vp
    keys = kp if held is None else held
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=kp.device)
    at = 0
    for i, (s, t) in enumerate(lens):
        if s == 0:
            continue
        w = case["window"] or t
        lo = max(0, t - s - w + 1)
        ids = torch.tensor(table[i][lo // page:(t - 1) // page + 1], device=kp.device)
        pos = torch.arange(t - s, t, device=kp.device)
        if case["op"] == "step":
            q = _exact_rows(st["q"][at:at + s], st["qw"], st, pos, nq)
        else:
            q = st["q"][at:at + s].double().reshape(s, nq, d)
        j = torch.arange(lo, t, device=kp.device)
        off = lo - lo // page * page
        for h in range(nkv):
            k = keys[ids, h].reshape(-1, d)[off:off + t - lo]
            v = vp[ids, h].reshape(-1, d)[off:off + t - lo]
            for a in range(h * (nq // nkv), (h + 1) * (nq // nkv)):
                z = (q[:, a] @ k.T) * d ** -0.5
                if case["softcap"]:
                    z = (z / case["softcap"]).tanh() * case["softcap"]
                seen = (j <= pos[:, None]) & (j > pos[:, None] - w)
                z = torch.where(seen, z, -math.inf)
                top = torch.logsumexp(z, -1, keepdim=True)
                if st["sink"] is not None:
                    top = torch.logaddexp(top, st["sink"][a].double().expand_as(top))
                out[at:at + s, a * d:(a + 1) * d] = (z - top).exp() @ v
        at += s
    return out if held is None else (out, kp, vp)
