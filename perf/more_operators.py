"""Cases and plain forms of the operators on a paged cache held in 4 bits.

Four operators: ``write`` appends new keys and values to the pages as codes and scales, the keys
normed and turned on the way, and reads the new rows back; ``read`` reads rows of the cache back;
``attend`` is the attention of a ragged batch of new tokens over the cache; ``step`` is the whole
step (norm, rotation, append, attention) with the new rows read back.

The cache: a row of D elements is D / 2 bytes, element 2 i in the low four bits of byte i, and a
bf16 scale for every 32 elements; a code c stands for (c - 8) * scale.  A row is written with
scale = max |x| / 7, rounded up to five significant bits, and c = 8 + round(x / scale).

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
GROUP = 32  # elements that share a scale


# ---------------------------------------------------------------------------- cases


def _case(op, lens, nq, nkv, d, dtype, page, window=0, softcap=0.0, sink=False, rd=0, interleaved=False, norm=True):
    """lens: "S:T" per sequence, S new tokens (or rows to read) ending at length T."""
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

    # one decode step's new rows of 64 sequences, into 64 different pages and back
    add("write-decode", _case("write", [(1, t) for t in _spread(64, 256, 2048, 11)], 32, 8, 128, BF16, 16))
    # ragged prompt chunks, one sequence without new tokens, one of a single token
    add("write-chunks", _case("write", [(512, 512), (512, 1813), (131, 700), (0, 400), (512, 2048), (509, 1021), (1, 1),
                                        (512, 1536)], 32, 8, 128, BF16, 64))
    # the last rows of one short sequence, as fp32
    add("read-small", _case("read", [(61, 131)], 64, 8, 64, F32, 16))
    # whole prefixes handed over to a cache of another type: every row of 8 sequences
    add("read-prefixes", _case("read", [(t, t) for t in _spread(8, 1024, 16384, 12)], 32, 8, 128, BF16, 16))
    # one token of one short sequence: latency alone
    add("attend-one", _case("attend", [(1, 131)], 32, 8, 128, BF16, 16))
    # the long-context decode batch: 64 ragged sequences, every key visible
    add("attend-decode", _case("attend", [(1, t) for t in _spread(64, 4096, 32768, 13)], 32, 8, 128, BF16, 16))
    # speculative verification: 8 drafted tokens for each of 16 sequences, windowed and capped
    add("attend-verify", _case("attend", [(8, t) for t in _spread(16, 6008, 6072, 14)], 32, 8, 128, BF16, 32,
                               window=4096, softcap=30.0))
    # chunked prefill: 512 tokens of each of 8 long windowed sequences
    add("attend-prefill", _case("attend", [(512, t) for t in _spread(8, 4608, 32768, 15)], 32, 8, 128, BF16, 64,
                                window=4096))
    # continuous batching: decoding sequences, two prompt chunks and two idle sequences in one call
    add("attend-mixed", _case("attend", [(1, t) for t in _spread(20, 128, 8192, 16)] + [(512, 4000), (333, 333), (0, 77),
                                                                                        (0, 0)],
                              64, 8, 64, BF16, 128, sink=True))
    # decode of fp32 rows
    add("attend-f32", _case("attend", [(1, 8192), (1, 2047), (1, 513), (1, 5000)], 64, 8, 64, F32, 16))
    # a whole decode step: norm, rotation, append, attention
    add("step-decode", _case("step", [(1, t) for t in _spread(32, 512, 4096, 17)], 32, 8, 128, BF16, 16))
    # a whole prompt step: a 2048-token prompt from an empty cache, and a short one behind it
    add("step-prompt", _case("step", [(2048, 2048), (77, 1077)], 32, 8, 128, BF16, 64))
    return cases


_HEADS = [(32, 8), (64, 8), (16, 16), (16, 2), (8, 1), (28, 4), (12, 4), (10, 2), (7, 1), (40, 8)]


def _logint(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "step"])
    dtype = BF16 if rng.random() < 0.75 else F32
    nq, nkv = rng.choice(_HEADS)
    d = rng.choice([64, 128, 128, 256] if dtype == BF16 else [32, 64, 128])
    rd = rng.choice([d, d, d // 2])
    inter = rng.random() < 0.3
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["decode", "verify", "chunks", "mixed"])
    n = _logint(rng, 1, 64 if kind == "decode" else 16)
    top = _logint(rng, 64, 16384)
    cap = 262144 if op == "attend" else 49152  # cache tokens in all
    room = 2.5e11  # products of queries and keys, and of weights and values
    lens = []
    for i in range(n):
        t = _logint(rng, max(1, top // 8), top)
        if op == "read":
            s = rng.choice([t, t, rng.randint(0, t)])
        elif kind == "decode":
            s = 1
        elif kind == "verify":
            s = rng.randint(1, 8)
        elif kind == "chunks":
            s = _logint(rng, 1, 1024)
        else:
            s = rng.choice([0, 1, 1, 1, 1, _logint(rng, 1, 512)])
        s = min(max(s, 0 if lens else 1), t)  # the first sequence has a token
        if dtype == F32 and op != "read":  # fewer new tokens: 32-bit products run at a fraction of the 16-bit rate
            s = min(s, 128)
        room -= 4.0 * s * t * nq * d
        if lens and (sum(x[1] for x in lens) + t > cap or room < 0):
            break
        lens.append((s, t))
    window = rng.choice([0, 0, _logint(rng, 16, 4096)])
    softcap = rng.choice([0.0, 0.0, 30.0])
    return _case(op, lens, nq, nkv, d, dtype, page, window, softcap, rng.random() < 0.3, rd, inter, rng.random() < 0.7)


# ---------------------------------------------------------------------------- inputs


def _lens(case):
    return [tuple(int(v) for v in w.split(":")) for w in case["lens"].split()]


def _tables(rows, rd, dtype, dev):
    """cos and sin of pos * THETA^(-2i/rd), angles in 64 bits, rounded once."""
    inv = THETA ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=dev) / rd)
    ang = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * inv[None, :]
    return torch.cos(ang).to(dtype).contiguous(), torch.sin(ang).to(dtype).contiguous()


def _quantise(x):
    """x (..., D) fp32 -> codes (..., D / 2) uint8, scales (..., D / 32) fp32 that bf16 holds exactly."""
    g = x.unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1)
    # up to four stored mantissa bits: the other 19 of the 23, rounded up (a quotient of tensors, since one
    # by a number is a product with its rounded reciprocal, and a multiple of 7 would go a step too high)
    s = (((top / torch.full_like(top, 7.0)).view(torch.int32) + 0x7FFFF) & ~0x7FFFF).view(torch.float32)
    s = torch.where(torch.isfinite(top), s, torch.nan)
    c = torch.round(g / s[..., None]).clamp(-7, 7)
    c = torch.where(torch.isnan(c), 0.0, c).flatten(-2).to(torch.int32) + 8
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8), s


def _values(codes, scales):
    """What codes (..., D / 2) and scales (..., D / 32) stand for, fp32 (..., D)."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8.0
    return (c.unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    lens, page = _lens(case), case["page"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def cache(pages):  # rows as the append left them, a fraction of the pages at a time
        codes = torch.empty(pages, nkv, page, d // 2, dtype=torch.uint8, device=dev)
        scales = torch.empty(pages, nkv, page, d // GROUP, dtype=torch.bfloat16, device=dev)
        step = max(1, (1 << 28) // (nkv * page * d))
        for a in range(0, pages, step):
            codes[a:a + step], scales[a:a + step] = _quantise(normal(min(step, pages - a), nkv, page, d))
        return codes, scales

    st = {"case": case}
    b, n = len(lens), sum(s for s, _ in lens)
    need = [(t + page - 1) // page for _, t in lens]
    width = max(1, max(need))
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
    st["kc"], st["ks"] = cache(pages)
    st["vc"], st["vs"] = cache(pages)
    turn, attends, new = case["op"] in ("write", "step"), case["op"] in ("attend", "step"), case["op"] != "attend"
    st["q"] = normal(n, nq * d).to(dt) if attends else None
    st["out"] = torch.zeros(n, nq * d, dtype=dt, device=dev) if attends else None
    st["k"], st["v"] = (normal(n, nkv * d).to(dt), normal(n, nkv * d).to(dt)) if turn else (None, None)
    st["ko"], st["vo"] = (torch.zeros(n, nkv * d, dtype=dt, device=dev) for _ in "kv") if new else (None, None)
    st["sink"] = normal(nq) if case["sink"] else None
    for name in ("qw", "kw"):
        w = (1.0 + 0.1 * normal(d)).to(dt)
        st[name] = w if turn and case["norm"] else None
    max_len = max(t for _, t in lens)
    st["cos"], st["sin"] = _tables(max_len, case["rd"], dt, dev) if turn else (None, None)
    # where each new row lies in the cache
    st["seq"] = torch.cat([torch.full((s,), i, device=dev) for i, (s, _) in enumerate(lens)]).long()
    st["pos"] = torch.cat([torch.arange(t - s, t, device=dev) for s, t in lens]).long()
    if own:
        from sliding_window_gqa_02_gb300 import gqaw

        def args(ws):
            return gqaw.make_paged_i4_args(
                st["q"], st["k"], st["v"], st["kc"], st["vc"], st["ks"], st["vs"], table, st["starts"], st["seqlens"],
                max(s for s, _ in lens), max_len, nq, nkv, st["out"], key_out=st["ko"], value_out=st["vo"], workspace=ws,
                local_window_size=case["window"], softcap=case["softcap"], head_sink=st["sink"],
                query_weight=st["qw"], key_weight=st["kw"], norm_eps=EPS, cos_cache=st["cos"], sin_cache=st["sin"],
                rotary_interleaved=case["interleaved"], dtype=dt)

        st["ws"] = gqaw.new_paged_i4_workspace(args(None), dev, torch.cuda.current_stream().cuda_stream)
        st["args"] = args(st["ws"])
    return st


# ---------------------------------------------------------------------------- plain forms (32 bits)


def _norm_turn(x, w, cos, sin, pos, rd, interleaved):
    """x (N, H, D) fp32: RMS norm over D times w (its factor in 64 bits: codes lie next to borders),
    then the first rd dimensions turned."""
    if w is not None:
        r = 1.0 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + EPS)
        x = x * r.float() * w.float()
    c, s = cos[pos].float()[:, None, :], sin[pos].float()[:, None, :]
    out = x.clone()
    if interleaved:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        out[..., 0:rd:2], out[..., 1:rd:2] = a * c - b * s, b * c + a * s
    else:
        h = rd // 2
        a, b = x[..., :h], x[..., h:rd]
        out[..., :h], out[..., h:rd] = a * c - b * s, b * c + a * s
    return out


def _plain_append(st):
    case = st["case"]
    nkv, d, page, pos = case["nkv"], case["d"], case["page"], st["pos"]
    k = _norm_turn(st["k"].view(-1, nkv, d).float(), st["kw"], st["cos"], st["sin"], pos, case["rd"], case["interleaved"])
    p, r = st["table"][st["seq"], pos // page].long(), pos % page
    for x, codes, scales in ((k, st["kc"], st["ks"]), (st["v"].view(-1, nkv, d).float(), st["vc"], st["vs"])):
        c, s = _quantise(x)
        codes[p, :, r] = c
        scales[p, :, r] = s.to(scales.dtype)


def _plain_read(st):
    page, pos = st["case"]["page"], st["pos"]
    p, r = st["table"][st["seq"], pos // page].long(), pos % page
    st["ko"].copy_(_values(st["kc"][p, :, r], st["ks"][p, :, r]).flatten(1))
    st["vo"].copy_(_values(st["vc"][p, :, r], st["vs"][p, :, r]).flatten(1))


def _plain_attend(st, q):
    """q (N, Nq, D) fp32 against the cache; the rows go to st["out"].  Sequences with the same number
    of new tokens go together, their keys padded to the longest."""
    case = st["case"]
    nq, nkv, d, page, w = case["nq"], case["nkv"], case["d"], case["page"], case["window"]
    grp, dev, lens = nq // nkv, q.device, _lens(case)
    starts = [0]
    for s, _ in lens:
        starts.append(starts[-1] + s)
    for s in sorted({s for s, _ in lens if s}):
        of = [i for i, (x, _) in enumerate(lens) if x == s]
        length = torch.tensor([lens[i][1] for i in of], device=dev)
        first = torch.clamp(length - s - w + 1, min=0) // page if w else torch.zeros_like(length)  # first page
        most = int(max((lens[i][1] - 1) // page - (max(0, lens[i][1] - s - w + 1) // page if w else 0) + 1 for i in of))
        col = torch.clamp(first[:, None] + torch.arange(most, device=dev), max=st["table"].shape[1] - 1)
        ids = torch.clamp(st["table"][torch.tensor(of, device=dev)[:, None], col].long(), min=0)
        k, v = (_values(c[ids], x[ids]).transpose(1, 2).reshape(len(of), nkv, most * page, d)
                for c, x in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
        key = (first * page)[:, None] + torch.arange(most * page, device=dev)
        rows = torch.tensor([starts[i] for i in of], device=dev)[:, None] + torch.arange(s, device=dev)
        at = (length - s)[:, None] + torch.arange(s, device=dev)
        for r0 in range(0, s, 512):
            r1 = min(s, r0 + 512)
            n = r1 - r0
            qq = q[rows[:, r0:r1]].view(len(of), n, nkv, grp, d).permute(0, 2, 3, 1, 4).reshape(len(of), nkv, grp * n, d)
            z = torch.matmul(qq, k.transpose(2, 3)).view(len(of), nkv, grp, n, -1) / math.sqrt(d)
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            a, j = at[:, r0:r1, None], key[:, None, :]
            hide = (j > a) | (j <= a - w) if w else j > a
            z = z.masked_fill(hide[:, None, None], float("-inf"))
            m = z.amax(-1, keepdim=True)
            if st["sink"] is not None:
                sk = st["sink"].view(nkv, grp, 1, 1)
                m = torch.maximum(m, sk)
            e = torch.exp(z - m)
            den = e.sum(-1, keepdim=True)
            if st["sink"] is not None:
                den = den + torch.exp(sk - m)
            o = torch.matmul((e / den).view(len(of), nkv, grp * n, -1), v).view(len(of), nkv, grp, n, d)
            st["out"][rows[:, r0:r1].flatten()] = o.permute(0, 3, 1, 2, 4).reshape(-1, nq * d).to(st["out"].dtype)


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if own:
        from sliding_window_gqa_02_gb300 import gqaw

        stream = torch.cuda.current_stream().cuda_stream
        if op == "write":
            gqaw.check(gqaw.gqaw_paged_i4_append(st["args"], stream))
        elif op == "attend":
            gqaw.check(gqaw.gqaw_paged_i4_attend(st["args"], stream))
            return st["out"]
        elif op == "step":
            gqaw.check(gqaw.gqaw_paged_i4_step(st["args"], stream))
        gqaw.check(gqaw.gqaw_paged_i4_read(st["args"], stream))
    else:
        if op in ("write", "step"):
            _plain_append(st)
        if op in ("attend", "step"):
            q = st["q"].view(-1, case["nq"], case["d"]).float()
            if op == "step":
                q = _norm_turn(q, st["qw"], st["cos"], st["sin"], st["pos"], case["rd"], case["interleaved"])
            _plain_attend(st, q)
        if op == "attend":
            return st["out"]
        _plain_read(st)
    if op == "read":
        return st["ko"], st["vo"]
    if op == "write":
        return st["ko"], st["vo"], st["ks"], st["vs"]
    return st["out"], st["ko"], st["vo"], st["ks"], st["vs"]


# ---------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    nq, nkv, d = case["nq"], case["nkv"], case["d"]
    es = 2 if case["dtype"] == BF16 else 4
    lens, w = _lens(case), case["window"]
    n = sum(s for s, _ in lens)
    held = d // 2 + d // GROUP * 2  # bytes of a row in the cache
    index = 4 * (2 * len(lens) + 1)
    op = case["op"]
    out = {"bytes": index, "flops": 0}
    if op in ("write", "step"):  # key and value rows in, codes and scales out; a row of the tables each
        out["bytes"] += n * nkv * (d * es + held) * 2 + n * (4 + case["rd"] * es)
        out["flops"] += n * nkv * (11 * d + 3 * case["rd"])
    if op != "attend":  # read back
        out["bytes"] += n * nkv * (d * es + (held if op == "read" else 0)) * 2
        out["flops"] += n * nkv * 4 * d
    if op in ("attend", "step"):
        rows = pairs = 0
        for s, t in lens:
            if s == 0:
                continue
            lo = max(0, t - s - w + 1) if w else 0
            rows += t - lo - (s if op == "step" else 0)  # a step's own rows are in hand
            pairs += sum(min(i + 1, w) if w else i + 1 for i in range(t - s, t))
            out["bytes"] += 4 * ((t - 1) // case["page"] - lo // case["page"] + 1)
        out["bytes"] += rows * nkv * held * 2 + 2 * n * nq * d * es
        out["flops"] += 4 * pairs * nq * d
    if op == "step":
        out["flops"] += n * nq * (4 * d + 3 * case["rd"])
    return out


# ---------------------------------------------------------------------------- the definition (64 bits)


def _exact_rows(x, w, st, heads):
    """Rows of x (N, heads * D), normed and turned, in float64: the turn as a complex product."""
    case = st["case"]
    d, rd = case["d"], case["rd"]
    y = x.double().reshape(x.shape[0], heads, d)
    if w is not None:
        y = y * w.double() / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
    turn = torch.complex(st["cos"].double(), st["sin"].double())[st["pos"]].unsqueeze(1)
    head, rest = y[..., :rd], y[..., rd:]
    if case["interleaved"]:
        z = torch.view_as_complex(head.reshape(x.shape[0], heads, rd // 2, 2).contiguous()) * turn
        head = torch.view_as_real(z).reshape(x.shape[0], heads, rd)
    else:
        z = torch.complex(head[..., :rd // 2].contiguous(), head[..., rd // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, rest], -1)


def _exact_held(y):
    """(what the cache holds of rows y (..., D) float64, its scales)."""
    parts = y.reshape(*y.shape[:-1], y.shape[-1] // GROUP, GROUP)
    top = parts.abs().amax(-1)
    mant, exp2 = torch.frexp(top / torch.full_like(top, 7))  # mant in [1/2, 1): five bits are multiples of 1/32
    s = torch.ldexp((mant * 32).ceil() / 32, exp2)
    n = torch.where(s[..., None] > 0, parts / s[..., None], 0.0).round()
    return (n * s[..., None]).reshape(y.shape), s


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    nq, nkv, d, page, op = case["nq"], case["nkv"], case["d"], case["page"], case["op"]
    lens = _lens(case)

    def rows_of(codes, scales, i, lo, hi, h):
        """Rows [lo, hi) of sequence i and head h, float64: nibbles by division."""
        j = torch.arange(lo, hi, device=codes.device)
        p = st["table"][i][j // page].long()
        byte = codes[p, h, j % page].int()
        nib = torch.empty(hi - lo, d, dtype=torch.float64, device=codes.device)
        nib[:, 0::2], nib[:, 1::2] = (byte % 16).double(), (byte // 16).double()
        return (nib - 8) * scales[p, h, j % page].double().repeat_interleave(GROUP, -1)

    new, scales = {}, {}
    if op in ("write", "step"):
        for name, y in (("k", _exact_rows(st["k"], st["kw"], st, nkv)), ("v", st["v"].double().reshape(-1, nkv, d))):
            new[name], s = _exact_held(y)
            scales[name] = st[name + "s"].double()
            scales[name][st["table"][st["seq"], st["pos"] // page].long(), :, st["pos"] % page] = s
    elif op == "read":
        for name in "kv":
            new[name] = torch.cat([torch.stack([rows_of(st[name + "c"], st[name + "s"], i, t - s, t, h) for h in range(nkv)], 1)
                                   for i, (s, t) in enumerate(lens)])
    flat = [new[x].reshape(-1, nkv * d) for x in "kv" if new]
    if op == "read":
        return tuple(flat)
    if op == "write":
        return (*flat, scales["k"], scales["v"])
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=st["out"].device)
    query = _exact_rows(st["q"], st["qw"], st, nq) if op == "step" else st["q"].double().reshape(-1, nq, d)
    at = 0
    for i, (s, t) in enumerate(lens):
        if s == 0:
            continue
        w = case["window"] or t
        lo = max(0, t - s - w + 1)
        pos, j = torch.arange(t - s, t, device=out.device), torch.arange(lo, t, device=out.device)
        seen = (j <= pos[:, None]) & (j > pos[:, None] - w)
        for h in range(nkv):
            if op == "step":  # the new rows as the append holds them
                k, v = (torch.cat([rows_of(st[x + "c"], st[x + "s"], i, lo, t - s, h) if t - s > lo else new[x][:0, h],
                                   new[x][at:at + s, h][max(0, lo - (t - s)):]]) for x in "kv")
            else:
                k, v = (rows_of(st[x + "c"], st[x + "s"], i, lo, t, h) for x in "kv")
            for a in range(h * (nq // nkv), (h + 1) * (nq // nkv)):
                z = (query[at:at + s, a] @ k.T) * d ** -0.5
                if case["softcap"]:
                    z = (z / case["softcap"]).tanh() * case["softcap"]
                z = torch.where(seen, z, -math.inf)
                top = torch.logsumexp(z, -1, keepdim=True)
                if st["sink"] is not None:
                    top = torch.logaddexp(top, st["sink"][a].double().expand_as(top))
                out[at:at + s, a * d:(a + 1) * d] = (z - top).exp() @ v
        at += s
    return out if op == "attend" else (out, *flat, scales["k"], scales["v"])
