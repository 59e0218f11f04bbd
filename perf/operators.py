"""Workloads of the paged NVFP4 key/value cache: block tables and slot maps
(``kv_tables``), the quantising append (``kv_append``) and attention over the
cache (``kv_attention``), each as the framework's call and in a plain form of
elementary torch operations.

A case is a dict of plain values.  Request lengths follow from the case alone
(``lens``), everything else from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ---------------------------------------------------------------------

def listed():
    """Head shapes: 32 query / 8 kv heads of 128 (the 8B layer: q 4096 of its
    6144 qkv outputs) and 64 / 8 of 128 (the 32B layer: 8192 of 10240), and
    generic ones of 64."""
    return [
        # one decode step of the largest batch of the small-M linears
        dict(name="tables_step", op="tables", reqs=8, new_lo=1, new_hi=1, past_lo=100, past_hi=4000,
             page=16, blocks=512, lens=1),
        # a large server step: decoding requests mixed with prompts being admitted
        dict(name="tables_mixed", op="tables", reqs=1000, new_lo=1, new_hi=517, past_lo=0, past_hi=60000,
             page=64, blocks=1024, lens=2),
        # the keys and values of one decode step
        dict(name="append_step", op="append", tokens=8, hkv=8, dim=128, page=16, dtype="bf16", lens=3),
        # a long prompt's keys and values
        dict(name="append_prompt", op="append", tokens=16384, hkv=8, dim=128, page=64, dtype="bf16", lens=4),
        # one request, one token, a short context: latency
        dict(name="decode_one", op="attention", reqs=1, new_lo=1, new_hi=1, past_lo=1030, past_hi=1030,
             empty=0, hq=32, hkv=8, dim=128, page=16, window=0, dtype="bf16", lens=5),
        # a padded batch of FP32 activations (the linears' default type), two of its rows without a request
        dict(name="decode_ragged_fp32", op="attention", reqs=24, new_lo=1, new_hi=1, past_lo=0, past_hi=6000,
             empty=2, hq=32, hkv=8, dim=128, page=32, window=0, dtype="fp32", lens=6),
        # two very long contexts: the split over a long axis
        dict(name="decode_long", op="attention", reqs=2, new_lo=1, new_hi=1, past_lo=100000, past_hi=131071,
             empty=0, hq=64, hkv=8, dim=128, page=64, window=0, dtype="bf16", lens=7),
        # a full batch of ordinary contexts: the cache stream's bandwidth
        dict(name="decode_batch", op="attention", reqs=64, new_lo=1, new_hi=1, past_lo=6000, past_hi=8191,
             empty=0, hq=32, hkv=8, dim=128, page=64, window=0, dtype="bf16", lens=8),
        # a drafted run of tokens checked in one pass, sliding window, heads of 64
        dict(name="verify_window", op="attention", reqs=16, new_lo=3, new_hi=6, past_lo=700, past_hi=9000,
             empty=0, hq=32, hkv=4, dim=64, page=16, window=1024, dtype="bf16", lens=9),
        # one chunk of a long prompt
        dict(name="chunk", op="attention", reqs=1, new_lo=2048, new_hi=2048, past_lo=30001, past_hi=30001,
             empty=0, hq=32, hkv=8, dim=128, page=64, window=0, dtype="bf16", lens=10),
        # whole prompts of different lengths in one call
        dict(name="prompts", op="attention", reqs=4, new_lo=333, new_hi=4096, past_lo=0, past_hi=0,
             empty=0, hq=64, hkv=8, dim=128, page=32, window=0, dtype="bf16", lens=11),
        # short prompts in FP32, a group of seven heads
        dict(name="prompts_fp32", op="attention", reqs=3, new_lo=50, new_hi=700, past_lo=0, past_hi=40,
             empty=0, hq=14, hkv=2, dim=64, page=16, window=0, dtype="fp32", lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def draw(rng):
    seed = rng.randrange(1 << 30)
    kind = rng.choice(("tables", "append", "decode", "decode", "verify", "prompt", "prompt"))
    page = rng.choice((16, 32, 64, 128))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if kind == "tables":
        new = _log(rng, 1, 517)
        past = _log(rng, 1, 60000)
        return dict(op="tables", reqs=_log(rng, 1, 1000), new_lo=rng.randint(0, 1), new_hi=new,
                    past_lo=0, past_hi=past, page=page, blocks=-(-(past + new) // page) + rng.randint(0, 9),
                    lens=seed)
    if kind == "append":
        return dict(op="append", tokens=_log(rng, 1, 16384), hkv=rng.choice((1, 2, 4, 8)),
                    dim=rng.choice((64, 128)), page=page, dtype=dtype, lens=seed)
    hkv = rng.choice((1, 2, 4, 8))
    case = dict(op="attention", reqs=1, new_lo=1, new_hi=1, past_lo=0, past_hi=0, empty=0,
                hq=hkv * rng.choice((1, 3, 4, 5, 7, 8)), hkv=hkv, dim=rng.choice((64, 128)), page=page,
                window=rng.choice((0, 0, _log(rng, 1, 4096))), dtype=dtype, lens=seed)
    if kind == "decode":
        reqs = _log(rng, 1, 64)
        hi = _log(rng, 1, min(131071, 400000 // reqs))
        case.update(reqs=reqs, past_lo=rng.choice((0, hi // 2, hi)), past_hi=hi, empty=rng.randint(0, reqs // 8))
    elif kind == "verify":
        reqs = _log(rng, 1, 32)
        hi = _log(rng, 16, 200000 // reqs)
        new = rng.randint(2, 16)
        case.update(reqs=reqs, new_lo=rng.randint(1, new), new_hi=new, past_lo=hi // 3, past_hi=hi)
    else:
        reqs = _log(rng, 1, 3)
        new = _log(rng, 17, 1500)
        past = rng.choice((0, _log(rng, 1, 4000)))
        case.update(reqs=reqs, new_lo=max(1, new // 3), new_hi=new, past_lo=past // 2, past_hi=past)
    return case


def lengths(case):
    """(tokens already in the cache, new tokens) of each request, from the case alone."""
    rng = random.Random(case["lens"])
    past, new = [], []
    for i in range(case["reqs"]):
        past.append(_log(rng, max(1, case["past_lo"]), max(1, case["past_hi"])) if case["past_hi"] else 0)
        new.append(rng.randint(case["new_lo"], case["new_hi"]))
    if case["op"] == "attention":
        for i in range(case["empty"]):  # a padding row of a fixed-size batch: one query row, no tokens
            past[i] = -1
    return past, new


# ---- inputs ----------------------------------------------------------------------

def _e2m1_code(t):
    a = t.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
         + (a > 5.0))
    return c | (torch.signbit(t).to(torch.uint8) << 3)


def _quantise(t, g):
    """NVFP4 of t [..., D] float32 with tensor scale g: (codes [..., D/2], E4M3 scale bytes [..., D/16])."""
    b = t.unflatten(-1, (-1, 16))
    six = 6.0 * g
    sc = torch.where(six > 0, b.abs().amax(-1) / six, 0.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = (sc.float() * g).unsqueeze(-1)
    q = _e2m1_code(torch.where(s == 0, torch.copysign(torch.zeros_like(b), b), b / s)).flatten(-2)
    q = q.unflatten(-1, (-1, 2))
    return q[..., 0] | (q[..., 1] << 4), sc.view(torch.uint8)


def _fill(pool, slots, k, v, kg, vg, page, dim):
    """Writes the NVFP4 form of k, v [T, H, D] float32 into the pool at the slots (those below 0 nowhere).

    Bytes of one (page, head): K codes [page][D/2], V codes [page][D/2], K scales [page][D/16], V scales [page][D/16]."""
    pages, heads, _ = pool.shape
    keep = slots >= 0
    p, o = slots[keep] // page, slots[keep] % page
    half, block = dim // 2, dim // 16
    flat = pool.view(pages, heads, -1)
    kq, ks = _quantise(k[keep], kg)
    vq, vs = _quantise(v[keep], vg)
    at = 0
    for data, width in ((kq, half), (vq, half), (ks, block), (vs, block)):
        part = flat[:, :, at:at + page * width].unflatten(-1, (page, width))
        part[p, :, o] = data
        at += page * width
    return pool


def _values(gen, shape, dtype, heads_gain=True):
    """Gaussian values with a few channels that are larger throughout, as keys have."""
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if heads_gain:
        gain = torch.ones(shape[-2:], device="cuda")
        at = torch.randint(0, shape[-1], (shape[-2], 3), generator=gen, device="cuda")
        gain.scatter_(1, at, 5.0)
        t *= gain
    return t.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "tables":
        return _prepare_tables(case, gen)
    if case["op"] == "append":
        return _prepare_append(case, gen)
    return _prepare_attention(case, gen)


def _prepare_tables(case, gen):
    past, new = lengths(case)
    page, reqs = case["page"], case["reqs"]
    held = [-(-n // page) for n in past]
    fresh = [-(-(n + c) // page) - h for n, c, h in zip(past, new, held)]
    pages = sum(held) + sum(fresh) + 100
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    kv_len = torch.tensor(past, dtype=torch.int32, device="cuda")
    held_d = torch.tensor(held, dtype=torch.int64, device="cuda")
    cols = torch.arange(case["blocks"], device="cuda")
    # what each request holds already; entries not given out yet are -1
    first = torch.cumsum(held_d, 0) - held_d
    at = (first[:, None] + cols).clamp(max=pages - 1)
    table = torch.where(cols < held_d[:, None], order[at], -1)
    return dict(case=case, kv_len=kv_len, q_len=torch.tensor(new, dtype=torch.int32, device="cuda"),
                free=order[sum(held):].clone(), head=torch.full((1,), 3, dtype=torch.int32, device="cuda"),
                table=table.to(torch.int32).contiguous(), tokens=sum(new))


def _pool(case, pages, gen):
    """Pages in use before: whatever they held is still there."""
    size = case["page"] * case["dim"] * 9 // 8
    return torch.randint(0, 120, (pages, case["hkv"], size), generator=gen, device="cuda", dtype=torch.uint8)


def _scales(k, v):
    return [(t.abs().max().float() / 2688.0).reshape(1) for t in (k, v)]


def _handle(state):
    """The framework's handle on the state's pool (what a program makes once)."""
    if own:
        import nvfp4_w4a4_decode_gb300 as nv
        case = state["case"]
        state["cache"] = nv.KVCache(state["pool"], state["kg"], state["vg"], page_size=case["page"],
                                    head_dim=case["dim"])
    return state


def _prepare_append(case, gen):
    tokens, page = case["tokens"], case["page"]
    dtype = DTYPES[case["dtype"]]
    # keys and values as slices of the qkv linear's output rows
    kv = _values(gen, (tokens, 2 * case["hkv"], case["dim"]), dtype)
    k, v = kv[:, :case["hkv"]], kv[:, case["hkv"]:]
    pages = -(-tokens // page) + 64
    if tokens > 64:  # a prompt: runs of a page each
        first = torch.randperm(pages, generator=gen, device="cuda")[:-(-tokens // page)] * page
        slots = (first[:, None] + torch.arange(page, device="cuda")).flatten()[:tokens]
    else:            # a decode step: one token of each request
        first = torch.randperm(pages, generator=gen, device="cuda")[:tokens] * page
        slots = first + torch.randint(0, page, (tokens,), generator=gen, device="cuda")
    kg, vg = _scales(k, v)
    return _handle(dict(case=case, k=k, v=v, slots=slots.contiguous(), kg=kg, vg=vg, pool=_pool(case, pages, gen)))


def _prepare_attention(case, gen):
    past, new = lengths(case)
    page, dim, hkv = case["page"], case["dim"], case["hkv"]
    dtype = DTYPES[case["dtype"]]
    seq = [max(0, n + c) for n, c in zip(past, new)]
    need = [-(-n // page) for n in seq]
    pages = sum(need) + 7
    blocks = max(1, max(need)) + 3
    order = torch.randperm(pages, generator=gen, device="cuda")
    need_d = torch.tensor(need, device="cuda")
    cols = torch.arange(blocks, device="cuda")
    first = torch.cumsum(need_d, 0) - need_d
    table = torch.where(cols < need_d[:, None], order[(first[:, None] + cols).clamp(max=pages - 1)], -1)
    pool = _pool(case, pages, gen)
    # the tokens of all requests, written a piece at a time
    seq_d = torch.tensor(seq, dtype=torch.int64, device="cuda")
    begin = torch.cumsum(seq_d, 0) - seq_d
    total = sum(seq)
    kg = vg = torch.full((1,), 25.0 / 2688.0, device="cuda")
    for at in range(0, total, 1 << 17):
        t = torch.arange(at, min(total, at + (1 << 17)), device="cuda")
        r = torch.searchsorted(begin, t, right=True) - 1
        i = t - begin[r]
        slots = table[r, i // page] * page + i % page
        k, v = _values(gen, (len(t), hkv, dim), torch.float32), _values(gen, (len(t), hkv, dim), torch.float32, False)
        _fill(pool, slots, k, v, kg, vg, page, dim)
    tokens = sum(new)
    q_start = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    # the queries as a slice of the qkv linear's output rows
    qkv = _values(gen, (tokens, case["hq"] + 2 * hkv, dim), dtype, False)
    return _handle(dict(case=case, q=qkv[:, :case["hq"]], pool=pool, table=table.to(torch.int32).contiguous(),
                        seq_len=seq_d.to(torch.int32), q_start=q_start, max_q=max(new), kg=kg, vg=vg))


# ---- one pass ----------------------------------------------------------------------

def run(state):
    if own:
        import nvfp4_w4a4_decode_gb300 as nv
        case = state["case"]
        if case["op"] == "tables":
            t = nv.kv_tables(state["kv_len"], state["q_len"], state["free"], state["head"], state["table"],
                             page_size=case["page"], tokens=state["tokens"])
            return dict(table=state["table"], seq_len=t.seq_len, q_start=t.q_start, slots=t.slots,
                        positions=t.positions, head=t.free_head)
        if case["op"] == "append":
            nv.kv_append(state["cache"], state["k"], state["v"], state["slots"])
            return state["pool"]
        out, lse = nv.kv_attention(state["cache"], state["q"], state["table"], state["seq_len"],
                                   state["q_start"], max_q=state["max_q"], window=case["window"],
                                   out_dtype=DTYPES[case["dtype"]], return_lse=True)
        return dict(out=out, lse=lse)
    plain = {"tables": _plain_tables, "append": _plain_append, "attention": _plain_attention}
    return plain[state["case"]["op"]](state)


def _plain_tables(state):
    page, table = state["case"]["page"], state["table"]
    past, new = state["kv_len"].long(), state["q_len"].long()
    seq = past + new
    q_start = torch.zeros(len(new) + 1, dtype=torch.int64, device="cuda")
    q_start[1:] = torch.cumsum(new, 0)
    held = (past + page - 1) // page
    fresh = (seq + page - 1) // page - held
    first = torch.cumsum(fresh, 0) - fresh
    cols = torch.arange(table.shape[1], device="cuda")
    given = (cols >= held[:, None]) & (cols < (held + fresh)[:, None])
    take = (state["head"].long() + first[:, None] + cols - held[:, None]).clamp(0, len(state["free"]) - 1)
    table.copy_(torch.where(given, state["free"][take], table))
    t = torch.arange(state["tokens"], device="cuda")
    r = torch.searchsorted(q_start, t, right=True) - 1
    pos = past[r] + t - q_start[r]
    slots = table[r, pos // page].long() * page + pos % page
    return dict(table=table, seq_len=seq.to(torch.int32), q_start=q_start.to(torch.int32), slots=slots,
                positions=pos.to(torch.int32), head=state["head"] + fresh.sum().to(torch.int32))


def _plain_append(state):
    case = state["case"]
    return _fill(state["pool"], state["slots"], state["k"].float(), state["v"].float(), state["kg"], state["vg"],
                 case["page"], case["dim"])


def _decoded(part, scales, g):
    """Codes [..., D/2] and scale bytes [..., D/16] to float32 [..., D]."""
    grid = torch.tensor(E2M1, device="cuda")
    grid = torch.cat([grid, -grid])
    codes = torch.stack([part & 15, part >> 4], -1).flatten(-2).int()
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * g
    return (grid[codes].unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _plain_attention(state):
    case, table, pool = state["case"], state["table"], state["pool"]
    page, dim, hkv, hq = case["page"], case["dim"], case["hkv"], case["hq"]
    half, block = dim // 2, dim // 16
    group, reqs, max_q = hq // hkv, case["reqs"], state["max_q"]
    seq = state["seq_len"].long()
    # [reqs, hkv, L, D] in float32, tokens past a request's end zeroed
    got = pool[table.clamp(min=0).long()].transpose(1, 2)
    cut = [page * half, page * half, page * block, page * block]
    kq, vq, ks, vs = (x.unflatten(-1, (page, -1)).flatten(2, 3) for x in got.split(cut, -1))
    there = torch.arange(kq.shape[2], device="cuda") < seq[:, None]
    zero = torch.zeros((), device="cuda")
    k = torch.where(there[:, None, :, None], _decoded(kq, ks, state["kg"]), zero)
    v = torch.where(there[:, None, :, None], _decoded(vq, vs, state["vg"]), zero)
    # queries [reqs, hkv, group * max_q, D], rows past a request's tokens repeat others and are dropped below
    start = state["q_start"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(max_q, device="cuda")
    rows = (start[:-1, None] + i).clamp(max=state["q"].shape[0] - 1)
    q = state["q"][rows].float().unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = torch.matmul(q, k.transpose(-1, -2)).unflatten(2, (group, max_q)) / math.sqrt(dim)
    j = torch.arange(k.shape[2], device="cuda")
    pos = (seq - count)[:, None] + i
    seen = (j <= pos[..., None]) & there[:, None]
    if case["window"]:
        seen &= j > pos[..., None] - case["window"]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, zero, m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (group, max_q)) / torch.where(l == 0, zero + 1, l)
    lse = (m + l.log()).squeeze(-1)
    t = torch.arange(state["q"].shape[0], device="cuda")
    r = torch.searchsorted(start, t, right=True) - 1
    at = t - start[r]
    out = o.permute(0, 3, 1, 2, 4)[r, at].flatten(1, 2)
    return dict(out=out.to(DTYPES[case["dtype"]]), lse=lse.permute(0, 3, 1, 2)[r, at].flatten(1, 2))


# ---- 64 bits --------------------------------------------------------------------------

def exact(case, seed):
    """Attention in float64, a request at a time.  The tables are whole
    numbers, and so are the appended bytes: each has one right value, fixed by
    rounding steps in 32 bits, which no computation in 64 bits repeats."""
    if case["op"] != "attention":
        return None
    state = prepare(case, seed)
    page, dim, hkv, hq, window = case["page"], case["dim"], case["hkv"], case["hq"], case["window"]
    seqs, starts = state["seq_len"].tolist(), state["q_start"].tolist()
    half, block = page * dim // 2, page * dim // 16
    grid = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device="cuda")
    out = torch.zeros((starts[-1], hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((starts[-1], hq), -math.inf, dtype=torch.float64, device="cuda")

    def rows(codes, scales, g, n):  # [n, D] of one head from its pages' bytes
        codes = codes.reshape(-1, dim // 2)[:n]
        x = torch.empty((n, dim), dtype=torch.float64, device="cuda")
        x[:, 0::2] = grid[(codes % 16).long()]
        x[:, 1::2] = grid[(codes // 16).long()]
        s = scales.reshape(-1, dim // 16)[:n].contiguous().view(torch.float8_e4m3fn).double()
        return x * s.repeat_interleave(16, -1) * g.double()

    for r, n in enumerate(seqs):
        a, b = starts[r], starts[r + 1]
        if n == 0 or a == b:
            continue
        mine = state["pool"][state["table"][r, :-(-n // page)].long()]
        key = torch.arange(n, device="cuda")
        for h in range(hkv):
            raw = mine[:, h]
            k = rows(raw[:, :half], raw[:, 2 * half:2 * half + block], state["kg"], n)
            v = rows(raw[:, half:2 * half], raw[:, 2 * half + block:], state["vg"], n)
            for g in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                for c in range(a, b, 1024):
                    e = min(b, c + 1024)
                    pos = n - (b - a) + torch.arange(c - a, e - a, device="cuda")[:, None]
                    hide = key > pos
                    if window:
                        hide |= key <= pos - window
                    s = (state["q"][c:e, g].double() @ k.T) * dim ** -0.5
                    s = s.masked_fill(hide, -math.inf)
                    some = ~hide.all(-1)
                    lse[c:e, g] = torch.logsumexp(s, -1)
                    out[c:e, g][some] = torch.softmax(s[some], -1) @ v
    return dict(out=out, lse=lse)


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    if case["op"] == "append":
        size = case["tokens"] * case["hkv"] * case["dim"]
        item = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * size * item + size * 9 // 8 + 8 * case["tokens"], "flops": 4 * size}
    past, new = lengths(case)
    if case["op"] == "tables":
        page = case["page"]
        fresh = sum(-(-(n + c) // page) - -(-n // page) for n, c in zip(past, new))
        # a token's page is read from the table where its request held it before
        return {"bytes": 16 * len(past) + 8 * fresh + 12 * sum(new) + 4 * len(past), "flops": 0}
    window = case["window"]
    tokens = pairs = 0
    for n, c in zip(past, new):
        seq = max(0, n + c)
        low = max(0, seq - c - window + 1) if window else 0
        tokens += seq - low
        for pos in range(seq - c, seq):
            pairs += min(pos + 1, window) if window else pos + 1
    item = 2 if case["dtype"] == "bf16" else 4
    rows = sum(new) * case["hq"]
    return {"bytes": tokens * case["hkv"] * case["dim"] * 9 // 8 + rows * (2 * case["dim"] * item + 4)
            + 4 * -(-tokens // case["page"]), "flops": 4 * case["dim"] * case["hq"] * pairs}
