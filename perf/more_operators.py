"""Workloads of three operators around the paged NVFP4 key/value cache: the
append with the position rotation applied on the way (``kv_append_rotary``),
attention of a batch whose requests share a prefix (``kv_attention_shared``) and
attention to the states of an encoder (``kv_cross_attention``), each as the
framework's call and in a plain form of elementary torch operations.

A case is a dict of plain values.  Request lengths follow from the case alone
(``lens``), everything else from the seed.

The pool is returned as the bytes it holds: the rotation's rounding steps are
fixed (two products and their difference, each rounded to float32), and so is
the block recipe behind it, so that every byte has one right value.
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
        # one decode step of the largest batch of the small-M linears: latency
        dict(name="rotary_step", op="rotary", reqs=8, new_lo=1, new_hi=1, past_lo=100, past_hi=4000, pad=0,
             hq=32, hkv=8, dim=128, rot=128, interleaved=False, page=16, dtype="bf16", lens=1),
        # a padded batch of FP32 activations (the linears' default type), half of each head rotated, in pairs
        # of neighbours
        dict(name="rotary_fp32", op="rotary", reqs=93, new_lo=1, new_hi=1, past_lo=0, past_hi=30000, pad=3,
             hq=14, hkv=2, dim=64, rot=32, interleaved=True, page=16, dtype="fp32", lens=2),
        # drafted tokens of a full batch, half of each head rotated
        dict(name="rotary_drafts", op="rotary", reqs=48, new_lo=3, new_hi=6, past_lo=700, past_hi=120000, pad=0,
             hq=64, hkv=8, dim=128, rot=64, interleaved=False, page=32, dtype="bf16", lens=3),
        # long prompts admitted together
        dict(name="rotary_prompts", op="rotary", reqs=5, new_lo=2500, new_hi=4096, past_lo=0, past_hi=0, pad=0,
             hq=32, hkv=8, dim=128, rot=128, interleaved=False, page=64, dtype="bf16", lens=4),
        # two answers of one short prompt, one token each: latency
        dict(name="shared_pair", op="shared", groups=1, reqs=2, prefix_lo=1030, prefix_hi=1030, past_lo=1,
             past_hi=60, new_lo=1, new_hi=1, empty=0, hq=32, hkv=8, dim=128, page=16, dtype="bf16", lens=5),
        # a full batch of short conversations behind one long system prompt, a token each
        dict(name="shared_batch", op="shared", groups=1, reqs=64, prefix_lo=8003, prefix_hi=8003, past_lo=30,
             past_hi=900, new_lo=1, new_hi=1, empty=0, hq=32, hkv=8, dim=128, page=64, dtype="bf16", lens=6),
        # sampled answers of a few prompts in FP32, three rows of the batch without a request
        dict(name="shared_samples_fp32", op="shared", groups=5, reqs=40, prefix_lo=200, prefix_hi=2500, past_lo=0,
             past_hi=500, new_lo=1, new_hi=1, empty=3, hq=14, hkv=2, dim=64, page=16, dtype="fp32", lens=7),
        # drafted tokens checked in one pass, three long documents behind them, heads of 64
        dict(name="shared_drafts", op="shared", groups=3, reqs=32, prefix_lo=6000, prefix_hi=30000, past_lo=0,
             past_hi=700, new_lo=3, new_hi=6, empty=0, hq=32, hkv=4, dim=64, page=16, dtype="bf16", lens=8),
        # questions of different lengths about one document, admitted together
        dict(name="shared_prompts", op="shared", groups=1, reqs=12, prefix_lo=12001, prefix_hi=12001, past_lo=0,
             past_hi=0, new_lo=150, new_hi=700, empty=0, hq=64, hkv=8, dim=128, page=32, dtype="bf16", lens=9),
        # a decoder's step on the states of an encoder, a kv head a query head
        dict(name="cross_step", op="cross", reqs=20, new_lo=1, new_hi=1, src_lo=300, src_hi=1500, empty=0,
             hq=16, hkv=16, dim=64, page=64, dtype="bf16", lens=10),
        # the beams of a few sources in FP32, one of them without states
        dict(name="cross_beams_fp32", op="cross", reqs=7, new_lo=4, new_hi=5, src_lo=1, src_hi=900, empty=1,
             hq=8, hkv=8, dim=64, page=16, dtype="fp32", lens=11),
        # target prefixes of different lengths on long sources
        dict(name="cross_targets", op="cross", reqs=8, new_lo=100, new_hi=448, src_lo=4000, src_hi=6000, empty=0,
             hq=32, hkv=8, dim=128, page=32, dtype="bf16", lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def draw(rng):
    seed = rng.randrange(1 << 30)
    kind = rng.choice(("rotary", "rotary", "decode", "decode", "drafts", "prompts", "cross", "cross"))
    dim = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 4, 8))
    case = dict(op=kind, reqs=1, new_lo=1, new_hi=1, hq=hkv * rng.choice((1, 3, 4, 5, 7, 8)), hkv=hkv, dim=dim,
                page=rng.choice((16, 32, 64, 128)), dtype=rng.choice(("bf16", "bf16", "fp32")), lens=seed)
    if kind == "rotary":
        tokens = _log(rng, 1, 16000)
        reqs = _log(rng, 1, min(tokens, 300))
        past = rng.choice((0, _log(rng, 1, 100000)))
        case.update(reqs=reqs, new_lo=max(1, tokens // reqs // 2), new_hi=tokens // reqs, past_lo=past // 3,
                    past_hi=past, pad=rng.choice((0, rng.randint(1, 9))),
                    rot=rng.choice((dim, dim, dim // 2, 32)), interleaved=rng.random() < 0.4)
        return case
    if kind == "cross":
        reqs = _log(rng, 1, 40)
        new = rng.choice((1, rng.randint(2, 8), _log(rng, 9, 1500) // reqs + 1))
        src = _log(rng, 1, min(20000, 150000 // reqs))
        case.update(reqs=reqs, new_lo=max(1, new // 3), new_hi=new, src_lo=rng.choice((1, max(1, src // 2))),
                    src_hi=src, empty=rng.randint(0, reqs // 8))
        if rng.random() < 0.4:
            case["hq"] = case["hkv"] = rng.choice((3, 6, 12, 16, 20))
        return case
    case.update(op="shared")
    if kind == "prompts":
        reqs = rng.randint(2, 12)
        new = _log(rng, 17, 3000 // reqs)
        prefix, past = _log(rng, 100, 10000), 0
        groups = rng.choice((1, 1, 2))
    else:
        reqs = _log(rng, 2, 64)
        new = 1 if kind == "decode" else rng.randint(2, 8)
        prefix = _log(rng, 100, 30000)
        past = _log(rng, 1, 100000 // reqs)
        groups = rng.randint(1, max(1, reqs // 4))
    prefix = min(prefix, 60000 // groups)
    case.update(groups=groups, reqs=reqs, prefix_lo=max(1, prefix // rng.choice((1, 4))), prefix_hi=prefix, past_lo=0,
                past_hi=past, new_lo=max(1, new // 2), new_hi=new, empty=rng.randint(0, reqs // 8))
    return case


def lengths(case):
    """Of each request, from the case alone: tokens before the new ones (behind the prefix where there is
    one, an encoder's states for cross attention; -1: a padding row of a fixed-size batch) and new
    tokens; of each group its prefix and how many requests it has."""
    rng = random.Random(case["lens"])
    lo, hi = (case["src_lo"], case["src_hi"]) if case["op"] == "cross" else (case["past_lo"], case["past_hi"])
    past, new, prefix, sizes = [], [], [], []
    for _ in range(case["reqs"]):
        past.append(_log(rng, max(1, lo), max(1, hi)) if hi else 0)
        new.append(rng.randint(case["new_lo"], case["new_hi"]))
    for i in range(case.get("empty", 0)):
        past[-1 - i] = -1
    if case["op"] == "shared":
        cuts = sorted(rng.sample(range(1, case["reqs"]), case["groups"] - 1))
        sizes = [b - a for a, b in zip([0] + cuts, cuts + [case["reqs"]])]
        prefix = [_log(rng, case["prefix_lo"], case["prefix_hi"]) for _ in sizes]
    return past, new, prefix, sizes


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


def _put(pool, at, width, page, p, o, data):
    """Writes rows of `width` bytes at tokens (p, o) of the part of every (page, head) that begins at byte `at`."""
    pool[:, :, at:at + page * width].unflatten(-1, (page, width))[p, :, o] = data


def _fill(pool, slots, k, v, kg, vg, page, dim):
    """Writes the NVFP4 form of k, v [T, H, D] float32 into the pool at the slots (those below 0 nowhere).

    Bytes of one (page, head): K codes [page][D/2], V codes [page][D/2], K scales [page][D/16], V scales [page][D/16]."""
    keep = slots >= 0
    p, o = slots[keep] // page, slots[keep] % page
    half, block = dim // 2, dim // 16
    kq, ks = _quantise(k[keep], kg)
    vq, vs = _quantise(v[keep], vg)
    _put(pool, 0, half, page, p, o, kq)
    _put(pool, page * half, half, page, p, o, vq)
    _put(pool, page * dim, block, page, p, o, ks)
    _put(pool, page * (dim + block), block, page, p, o, vs)
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


def _pool(case, pages, gen):
    """Pages in use before: whatever they held is still there."""
    size = case["page"] * case["dim"] * 9 // 8
    return torch.randint(0, 120, (pages, case["hkv"], size), generator=gen, device="cuda", dtype=torch.uint8)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _starts(counts):
    return _ints([sum(counts[:i]) for i in range(len(counts) + 1)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = _prepare_rotary(case, gen) if case["op"] == "rotary" else _prepare_attention(case, gen)
    return _handle(dict(state, case=case))


def _handle(state):
    """The framework's handle on the state's pool (what a program makes once)."""
    if own:
        import nvfp4_w4a4_decode_gb300 as nv
        case = state["case"]
        state["cache"] = nv.KVCache(state["pool"], state["kg"], state["vg"], page_size=case["page"],
                                    head_dim=case["dim"])
    return state


def _rotary_table(positions, rot, base=10000.0):
    """Float32 [positions][rot]: the cosines of a position's rot / 2 angles, then their sines."""
    freq = base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _prepare_rotary(case, gen):
    past, new, _, _ = lengths(case)
    page, dim, hkv, hq = case["page"], case["dim"], case["hkv"], case["hq"]
    dtype = DTYPES[case["dtype"]]
    tokens = sum(new) + case["pad"]
    # every request's new tokens on pages of its own
    first = [n // page for n in past]
    held = [(n + c - 1) // page - f + 1 for n, c, f in zip(past, new, first)]
    pages = sum(held) + 16
    order = torch.randperm(pages, generator=gen, device="cuda")
    count = _ints(new, torch.int64)
    r = torch.repeat_interleave(torch.arange(len(new), device="cuda"), count)
    pos = _ints(past, torch.int64)[r] + torch.arange(sum(new), device="cuda") - (torch.cumsum(count, 0) - count)[r]
    begin = _ints(held, torch.int64)
    begin = torch.cumsum(begin, 0) - begin
    slots = order[begin[r] + pos // page - _ints(first, torch.int64)[r]] * page + pos % page
    pad = torch.zeros(case["pad"], dtype=torch.int64, device="cuda")
    # queries, keys and values as slices of the qkv linear's output rows
    rows = _values(gen, (tokens, hq + 2 * hkv, dim), dtype)
    q, k, v = rows.split((hq, hkv, hkv), 1)
    kg = (k.abs().max().float() * 1.2 / 2688.0).reshape(1)  # a pair's length, which the rotation keeps
    vg = (v.abs().max().float() / 2688.0).reshape(1)
    return dict(q=q, k=k, v=v, slots=torch.cat([slots, pad - 1]), positions=torch.cat([pos, pad]).to(torch.int32),
                rotary=_rotary_table(max(n + c for n, c in zip(past, new)) + 1, case["rot"]), kg=kg, vg=vg,
                pool=_pool(case, pages, gen))


def _tables(spans, page, order, blocks):
    """Block tables [len(spans), blocks] int64 that hold the keys [lo, hi) of each span on pages of `order`
    (what lies before and behind is -1), and the pages used."""
    first = [lo // page for lo, hi in spans]
    need = [max(0, -(-hi // page) - f) if hi > lo else 0 for (lo, hi), f in zip(spans, first)]
    begin = _ints([sum(need[:i]) - f for i, f in enumerate(first)], torch.int64)[:, None]
    cols = torch.arange(blocks, device="cuda")
    first, need_d = _ints(first, torch.int64)[:, None], _ints(need, torch.int64)[:, None]
    there = (cols >= first) & (cols < first + need_d)
    return torch.where(there, order[(begin + cols).clamp(0, len(order) - 1)], -1), sum(need)


def _prepare_attention(case, gen):
    past, new, prefix, sizes = lengths(case)
    page, dim, hkv, hq = case["page"], case["dim"], case["hkv"], case["hq"]
    dtype = DTYPES[case["dtype"]]
    cross = case["op"] == "cross"
    shared = [n for n, s in zip(prefix, sizes) for _ in range(s)] or [0] * len(past)
    seq = [max(0, n) if cross else 0 if n < 0 else p + n + c for p, n, c in zip(shared, past, new)]
    spans = [(p, max(p, n)) if n else (0, 0) for p, n in zip(shared, seq)]
    pages = sum(-(-hi // page) - lo // page for lo, hi in spans) + sum(-(-n // page) for n in prefix) + 7
    order = torch.randperm(pages, generator=gen, device="cuda")
    table, used = _tables(spans, page, order, max(1, -(-max(seq) // page)) + 3)
    pool = _pool(case, pages, gen)
    state = dict(pool=pool, seq_len=_ints(seq), q_start=_starts(new), max_q=max(new),
                 kg=torch.full((1,), 25.0 / 2688.0, device="cuda"), vg=torch.full((1,), 25.0 / 2688.0, device="cuda"))
    parts = [(table, spans)]
    if prefix:
        own_spans = [(0, n) for n in prefix]
        prefix_table, _ = _tables(own_spans, page, order[used:], -(-max(prefix) // page) + 2)
        parts.append((prefix_table, own_spans))
        # sizes that a program knows: the most requests of a group, the most keys on a request's own pages
        state.update(prefix_table=prefix_table.to(torch.int32), prefix_len=_ints(prefix), group_start=_starts(sizes),
                     members=max(sizes),
                     own_keys=max(1, max(-(-hi // page) - lo // page for lo, hi in spans)) * page)
    for rows, runs in parts:  # the keys and values, written a piece at a time
        lo = _ints([a for a, b in runs], torch.int64)
        count = _ints([b for a, b in runs], torch.int64) - lo
        begin = torch.cumsum(count, 0) - count
        total = sum(b - a for a, b in runs)
        for at in range(0, total, 1 << 17):
            t = torch.arange(at, min(total, at + (1 << 17)), device="cuda")
            r = torch.searchsorted(begin, t, right=True) - 1
            i = t - begin[r] + lo[r]
            slots = rows[r, i // page] * page + i % page
            k, v = _values(gen, (len(t), hkv, dim), torch.float32), _values(gen, (len(t), hkv, dim), torch.float32, False)
            _fill(pool, slots, k, v, state["kg"], state["vg"], page, dim)
    # the queries as a slice of the qkv linear's output rows
    rows = _values(gen, (sum(new), hq + 2 * hkv, dim), dtype, False)
    return dict(state, q=rows[:, :hq], table=table.to(torch.int32).contiguous())


# ---- one pass ----------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        import nvfp4_w4a4_decode_gb300 as nv
        if case["op"] == "rotary":
            q = nv.kv_append_rotary(state["cache"], state["q"], state["k"], state["v"], state["slots"],
                                    state["positions"], state["rotary"], interleaved=case["interleaved"])
            return dict(q=q, pool=state["pool"])
        if case["op"] == "shared":
            out, lse = nv.kv_attention_shared(state["cache"], state["q"], state["prefix_table"], state["prefix_len"],
                                              state["table"], state["seq_len"], state["q_start"],
                                              group_start=state["group_start"], max_q=state["max_q"],
                                              return_lse=True)
        else:
            out, lse = nv.kv_cross_attention(state["cache"], state["q"], state["table"], state["seq_len"],
                                             state["q_start"], max_q=state["max_q"], return_lse=True)
        return dict(out=out, lse=lse)
    plain = {"rotary": _plain_rotary, "shared": _plain_shared, "cross": _plain_cross}
    return plain[case["op"]](state)


def _rotated(x, cos, sin, interleaved):
    """x [T, H, D] float32 with its first rot elements turned: pairs (i, i + rot / 2), or (2 i, 2 i + 1)."""
    half = cos.shape[-1]
    turn, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if interleaved else (turn[..., :half], turn[..., half:])
    c, s = cos[:, None], sin[:, None]
    a, b = a * c - b * s, b * c + a * s
    turn = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turn, rest], -1)


def _plain_rotary(state):
    case = state["case"]
    cos, sin = state["rotary"][state["positions"].long()].chunk(2, -1)
    q = _rotated(state["q"].float(), cos, sin, case["interleaved"])
    k = _rotated(state["k"].float(), cos, sin, case["interleaved"])
    pool = _fill(state["pool"], state["slots"], k, state["v"].float(), state["kg"], state["vg"], case["page"],
                 case["dim"])
    return dict(q=q.to(state["q"].dtype), pool=pool)


def _decoded(part, scales, g):
    """Codes [..., D/2] and scale bytes [..., D/16] to float32 [..., D]."""
    grid = torch.tensor(E2M1, device="cuda")
    grid = torch.cat([grid, -grid])
    codes = torch.stack([part & 15, part >> 4], -1).flatten(-2).int()
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * g
    return (grid[codes].unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _cached(state, table, there):
    """(K, V) float32 [rows of the table, hkv, blocks * page, D]; zeros where `there` [rows, blocks * page] is not."""
    page, dim = state["case"]["page"], state["case"]["dim"]
    half, block = page * dim // 2, page * dim // 16
    got = state["pool"][table.clamp(min=0).long()].transpose(1, 2)
    kq, vq, ks, vs = got.split([half, half, block, block], -1)
    k = _decoded(kq.unflatten(-1, (page, -1)).flatten(2, 3), ks.unflatten(-1, (page, -1)).flatten(2, 3), state["kg"])
    v = _decoded(vq.unflatten(-1, (page, -1)).flatten(2, 3), vs.unflatten(-1, (page, -1)).flatten(2, 3), state["vg"])
    zero = torch.zeros((), device="cuda")
    there = there[:, None, :, None]
    return torch.where(there, k, zero), torch.where(there, v, zero)


def _attend(q, k, v, seen):
    """Of queries [B, hkv, group, n, D] over keys [B, hkv, L, D] that rows see by seen [B, n, L]: the sum of
    exp(s - m) v, the sum of exp(s - m) and m."""
    group = q.shape[2]
    s = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (group, -1)) / math.sqrt(q.shape[-1])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    return torch.matmul(p.flatten(2, 3), v).unflatten(2, (group, -1)), p.sum(-1, keepdim=True), m


def _finish(state, o, l, m, pick):
    """The rows as the framework's call gives them, from [B, hkv, group, n, ...] by pick = (B, n) of each row."""
    out = (o / torch.where(l == 0, 1.0, l)).permute(0, 3, 1, 2, 4)[pick].flatten(1, 2)
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2)[pick].flatten(1, 2)
    return dict(out=out.to(state["q"].dtype), lse=lse)


def _rows(state):
    """Queries [reqs, hkv, group, max_q, D] float32 (rows past a request's tokens repeat others), each row's
    request and its place there, and the requests' rows."""
    case, start = state["case"], state["q_start"].long()
    i = torch.arange(state["max_q"], device="cuda")
    at = (start[:-1, None] + i).clamp(max=state["q"].shape[0] - 1)
    q = state["q"][at].float().unflatten(2, (case["hkv"], -1)).permute(0, 2, 3, 1, 4)
    t = torch.arange(state["q"].shape[0], device="cuda")
    r = torch.searchsorted(start, t, right=True) - 1
    return q, r, t - start[r], start[1:] - start[:-1]


def _plain_cross(state):
    seq = state["seq_len"].long()
    there = torch.arange(state["table"].shape[1] * state["case"]["page"], device="cuda") < seq[:, None]
    k, v = _cached(state, state["table"], there)
    q, r, at, _ = _rows(state)
    return _finish(state, *_attend(q, k, v, there[:, None].expand(-1, state["max_q"], -1)), (r, at))


def _plain_shared(state):
    """Every group's prefix against all rows of the group at once, the requests' own keys against their rows,
    and the two joined by their largest scores."""
    page = state["case"]["page"]
    seq, shared, bound = state["seq_len"].long(), state["prefix_len"].long(), state["group_start"].long()
    q, r, at, count = _rows(state)
    of = torch.searchsorted(bound, torch.arange(len(seq), device="cuda"), right=True) - 1
    # the requests of a group side by side [groups, members], the last of a smaller group again
    members = state["members"]
    side = (bound[:-1, None] + torch.arange(members, device="cuda")).minimum(bound[1:, None] - 1)
    qg = q[side].permute(0, 2, 3, 1, 4, 5).flatten(3, 4)
    there = torch.arange(state["prefix_table"].shape[1] * page, device="cuda") < shared[:, None]
    pre = _attend(qg, *_cached(state, state["prefix_table"], there), there[:, None].expand(-1, qg.shape[3], -1))
    place = torch.arange(len(seq), device="cuda") - bound[of]
    o1, l1, m1 = (x.unflatten(3, (members, -1)).permute(0, 3, 1, 2, 4, 5)[of, place] for x in pre)
    # the tokens behind the prefix, from the first page that holds one
    first = shared[of] // page
    j = first[:, None] * page + torch.arange(state["own_keys"], device="cuda")
    table = state["table"].gather(1, (j[:, ::page] // page).clamp(max=state["table"].shape[1] - 1))
    there = (j >= shared[of][:, None]) & (j < seq[:, None])
    pos = (seq - count)[:, None] + torch.arange(state["max_q"], device="cuda")
    seen = there[:, None] & (j[:, None] <= pos[..., None])
    o2, l2, m2 = _attend(q, *_cached(state, table, there), seen)
    m1 = torch.where((seq == 0)[:, None, None, None, None], -math.inf, m1)  # a request without tokens sees nothing
    m = torch.maximum(m1, m2)
    w1, w2 = (torch.exp(x - torch.where(m == -math.inf, 0.0, m)) for x in (m1, m2))
    return _finish(state, o1 * w1 + o2 * w2, l1 * w1 + l2 * w2, m, (r, at))


# ---- 64 bits --------------------------------------------------------------------------

def exact(case, seed):
    """Attention in float64, a request and a head at a time; the rotated queries in float64.  The pool's bytes
    have one right value each, fixed by rounding steps in 32 bits, which no computation in 64 bits repeats."""
    state = prepare(case, seed)
    if case["op"] == "rotary":
        rot, half = case["rot"], case["rot"] // 2
        angle = state["rotary"].double()[state["positions"].long()][:, None]
        turned = state["q"].double()
        one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
        z = torch.complex(turned[..., one], turned[..., two]) * torch.complex(angle[..., :half], angle[..., half:])
        turned[..., one], turned[..., two] = z.real, z.imag
        return dict(q=turned, pool=None)
    page, dim, hkv, hq = case["page"], case["dim"], case["hkv"], case["hq"]
    half, block = page * dim // 2, page * dim // 16
    grid = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device="cuda")
    starts, seqs = state["q_start"].tolist(), state["seq_len"].tolist()
    out = torch.zeros((starts[-1], hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((starts[-1], hq), -math.inf, dtype=torch.float64, device="cuda")

    def rows(raw, is_v, lo, hi):  # tokens [lo, hi) of one head, of its pages' bytes
        codes = raw[:, half:2 * half] if is_v else raw[:, :half]
        scales = raw[:, 2 * half + block:] if is_v else raw[:, 2 * half:2 * half + block]
        codes = codes.reshape(-1, dim // 2)[lo:hi]
        x = torch.empty((hi - lo, dim), dtype=torch.float64, device="cuda")
        x[:, 0::2] = grid[(codes % 16).long()]
        x[:, 1::2] = grid[(codes // 16).long()]
        s = scales.reshape(-1, dim // 16)[lo:hi].contiguous().view(torch.float8_e4m3fn).double()
        return x * s.repeat_interleave(16, -1) * (state["vg"] if is_v else state["kg"]).double()

    def tokens(table, lo, hi, h):  # K and V of keys [lo, hi)
        raw = state["pool"][table[lo // page:-(-hi // page)].long(), h]
        off = lo // page * page
        return rows(raw, False, lo - off, hi - off), rows(raw, True, lo - off, hi - off)

    if case["op"] == "shared":
        bound, prefix = state["group_start"].tolist(), state["prefix_len"].tolist()
    else:
        bound, prefix = list(range(len(seqs) + 1)), [0] * len(seqs)
    for g, p in enumerate(prefix):
        for h in range(hkv):
            k0, v0 = tokens(state["prefix_table"][g], 0, p, h) if p else (None, None)
            for r in range(bound[g], bound[g + 1]):
                n, a, b = seqs[r], starts[r], starts[r + 1]
                if n == 0 or a == b:
                    continue
                k, v = tokens(state["table"][r], p, n, h)
                if p:
                    k, v = torch.cat([k0, k]), torch.cat([v0, v])
                for i in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                    s = (state["q"][a:b, i].double() @ k.T) * dim ** -0.5
                    if case["op"] == "shared":
                        pos = n - (b - a) + torch.arange(b - a, device="cuda")[:, None]
                        s = s.masked_fill(torch.arange(n, device="cuda") > pos, -math.inf)
                    lse[a:b, i] = torch.logsumexp(s, -1)
                    out[a:b, i] = torch.softmax(s, -1) @ v
    return dict(out=out, lse=lse)


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    past, new, prefix, sizes = lengths(case)
    item = 2 if case["dtype"] == "bf16" else 4
    dim, hkv, hq = case["dim"], case["hkv"], case["hq"]
    if case["op"] == "rotary":
        tokens = sum(new)
        size = tokens * hkv * dim
        turned = tokens * (hq + hkv) * case["rot"]
        # q in and out, k and v in, codes and scales out, a row of the table, slot and position a token
        return {"bytes": 2 * (tokens + case["pad"]) * hq * dim * item + 2 * size * item + size * 9 // 8
                + tokens * 4 * case["rot"] + 12 * tokens, "flops": 3 * turned + 4 * size}
    shared = [n for n, s in zip(prefix, sizes) for _ in range(s)] or [0] * len(past)
    keys, pairs = sum(prefix), 0
    for p, n, c in zip(shared, past, new):
        if n < 0:
            continue
        keys += n + (c if case["op"] == "shared" else 0)
        pairs += c * (p + n) + (c * (c + 1) // 2 if case["op"] == "shared" else 0)
    rows = sum(new) * hq
    return {"bytes": keys * hkv * dim * 9 // 8 + rows * (2 * dim * item + 4) + 4 * -(-keys // case["page"]),
            "flops": 4 * dim * hq * pairs}
