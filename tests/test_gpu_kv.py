"""The paged NVFP4 cache on the GPU through the public entry points: block
tables against a loop over requests, appended bytes against the oracle's
quantiser, attention against its definition in 64 bits."""
import itertools
import math

import numpy as np
import pytest
import torch

import oracle
from kv_helpers import attention, check_attention, page_values

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def nv():
    import nvfp4_w4a4_decode_gb300 as nvmod
    from nvfp4_w4a4_decode_gb300 import build as nvbuild
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    nvbuild.build()
    oracle.build()
    nvmod.library()
    nvmod.device_status(clear=True)
    return nvmod


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


# ---- block tables ----------------------------------------------------------------

def tables_by_hand(past, new, page, free, head, table, tokens):
    """The header's definition, one request and one token at a time."""
    table = [list(row) for row in table]
    cap = len(table[0]) * page if table else 0
    seq, start, slots, positions = [], [0], [], []
    for r, (n, c) in enumerate(zip(past, new)):
        n, c = max(n, 0), max(c, 0)
        end = min(n + c, cap)
        held = -(-min(n, cap) // page)
        for b in range(held, -(-end // page)):
            table[r][b] = free[head] if 0 <= head < len(free) else -1
            head += 1
        for pos in range(n, n + c):
            p = table[r][pos // page] if pos < end else -1
            positions.append(pos)
            slots.append(p * page + pos % page if p >= 0 else -1)
        seq.append(end)
        start.append(start[-1] + c)
    pad = tokens - len(slots)
    return table, seq, start, (slots + [-1] * pad)[:tokens], (positions + [0] * pad)[:tokens], head


def run_tables(nv, past, new, page, blocks, free, head, tokens=None, table=None):
    tokens = sum(max(c, 0) for c in new) if tokens is None else tokens
    if table is None:
        table, nxt = [], 100000
        for n in past:
            held = -(-min(max(n, 0), blocks * page) // page)
            table.append([nxt + i if i < held else -7 for i in range(blocks)])
            nxt += held
    want = tables_by_hand(past, new, page, free, head, table, tokens)
    td = ints(table).reshape(len(past), blocks)
    args = (ints(past), ints(new), ints(free), ints([head]), td)
    for _ in range(2):  # the second call repeats the first
        got = nv.kv_tables(*args, page_size=page, tokens=tokens)
        assert td.tolist() == want[0]
        assert got.seq_len.tolist() == want[1]
        assert got.q_start.tolist() == want[2]
        assert got.slots.tolist() == want[3]
        assert got.positions.tolist() == want[4]
        assert got.free_head.tolist() == [want[5]]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("reqs,seed", [(1, 0), (7, 1), (513, 2), (1500, 3)])
def test_tables(nv, page, reqs, seed):
    rng = np.random.default_rng(seed + page)
    past = rng.integers(0, 5 * page, reqs).tolist()
    new = rng.integers(0, 2 * page if reqs < 100 else 9, reqs).tolist()
    past[0], new[-1] = 2 * page, page + 1            # a full last page, more than one new page
    nv.device_status(clear=True)
    run_tables(nv, past, new, page, 8, list(range(5, 5 + 8 * reqs)), 3)
    assert nv.device_status() == 0


def test_tables_edges(nv):
    nv.device_status(clear=True)
    run_tables(nv, [0, 0], [0, 0], 16, 4, [1, 2, 3], 0, tokens=0)       # nothing new
    run_tables(nv, [0, 0], [0, 0], 16, 4, [1, 2, 3], 0, tokens=5)       # only padding
    run_tables(nv, [15, 16, 17], [1, 1, 1], 16, 2, [9, 8], 0, tokens=8)  # page ends, padding
    run_tables(nv, [-3, 5], [2, -1], 16, 2, [9, 8], 0, tokens=4)        # negative counts as 0
    run_tables(nv, [], [], 16, 0, [4], 0, tokens=3, table=[])           # no requests
    assert nv.device_status() == 0


def test_tables_too_short_are_reported(nv):
    for past, new, blocks, free, head in (([0, 0], [40, 40], 4, [5, 6, 7, 8], 0),    # free list ends
                                          ([0], [20], 4, [5, 6, 7], -1),             # head below 0
                                          ([30, 100], [10, 4], 2, [5, 6, 7], 0)):    # table ends
        nv.device_status(clear=True)
        run_tables(nv, past, new, 16, blocks, free, head)
        assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
    nv.device_status(clear=True)
    run_tables(nv, [0, 3], [5, 5], 16, 2, [5, 6, 7], 0, tokens=7)  # fewer rows than new tokens
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE


def test_tables_largest(nv):
    reqs = 16384
    past = ints(np.arange(reqs) % 33)
    new = torch.ones(reqs, dtype=torch.int32, device="cuda")
    table = torch.full((reqs, 4), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(reqs, device="cuda") + 50000
    table[:, 1] = torch.arange(reqs, device="cuda") + 90000
    free = torch.randperm(reqs, device="cuda").to(torch.int32)
    got = nv.kv_tables(past, new, free, ints([0]), table, page_size=16, tokens=reqs)
    page = table.gather(1, (past // 16)[:, None].long())[:, 0]
    assert torch.equal(got.slots, page.long() * 16 + past % 16)
    assert got.free_head.item() == (past % 16 == 0).sum().item()
    assert torch.equal(got.q_start, torch.arange(reqs + 1, device="cuda", dtype=torch.int32))


# ---- append ----------------------------------------------------------------------

def make_cache(nv, pages, heads, dim, page, kg, vg, layers=1, layer=0, fill=None):
    """A cache over one layer of a pool of `layers` (strided pages)."""
    whole = nv.kv_pool(pages * layers, heads, dim, page)
    if fill is None:
        whole.random_(0, 256)
    else:
        whole.fill_(fill)
    pool = whole.view(pages, layers, heads, -1)[:, layer]
    return nv.KVCache(pool, kg, vg, page_size=page, head_dim=dim), whole


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("heads,dim,page,tokens,layers",
                         [(8, 128, 16, 1, 1), (8, 128, 64, 200, 2), (1, 64, 16, 37, 1),
                          (3, 64, 32, 65, 1), (5, 128, 128, 33, 3), (32, 128, 256, 40, 1)])
def test_append_bytes(nv, dtype, heads, dim, page, tokens, layers):
    gen = torch.Generator(device="cuda").manual_seed(heads * dim + page)
    rows = torch.randn((tokens, 3 * heads + 1, dim), generator=gen, device="cuda")
    # block scales from subnormal to saturated, blocks of zeros, signed zeros
    rows *= torch.exp2(torch.randint(-14, 4, (tokens, 3 * heads + 1, 1), generator=gen, device="cuda"))
    rows[::5, :, :16] = 0.0
    rows[1::5, :, :16] = -0.0
    rows = rows.to(dtype)
    k, v = rows[:, :heads], rows[:, heads:2 * heads]
    kg, vg = ints([0.0011], FP32), ints([0.0002], FP32)
    pages = -(-tokens // page) + 5
    cache, whole = make_cache(nv, pages, heads, dim, page, kg, vg, layers, layers - 1)
    before = whole.clone()
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:tokens].contiguous()
    slots[::7] = -1
    nv.device_status(clear=True)
    nv.kv_append(cache, k, v, slots)
    assert nv.device_status() == 0
    want = before.clone()
    mine = want.view(pages, layers, heads, -1)[:, layers - 1]
    half, block = page * dim // 2, page * dim // 16
    for part, (x, g) in enumerate(((k, kg), (v, vg))):
        q, s = oracle.quantize(x.float().cpu().numpy().reshape(tokens * heads, dim), np.float32(g.item()))
        q = torch.from_numpy(q).cuda().view(tokens, heads, -1)
        s = torch.from_numpy(s).cuda().view(tokens, heads, -1)
        for t in range(tokens):
            if slots[t] < 0:
                continue
            p, o = divmod(slots[t].item(), page)
            at = part * half + o * dim // 2
            mine[p, :, at:at + dim // 2] = q[t]
            at = 2 * half + part * block + o * dim // 16
            mine[p, :, at:at + dim // 16] = s[t]
    assert torch.equal(whole, want)


def test_append_bad_slots_are_skipped_and_reported(nv):
    kg = ints([0.01], FP32)
    cache, whole = make_cache(nv, 4, 2, 64, 16, kg, kg)
    before = whole.clone()
    k = torch.randn((5, 2, 64), device="cuda")
    nv.device_status(clear=True)
    nv.kv_append(cache, k, k, ints([64, -2, 1 << 40, -(1 << 40), -1], torch.int64))
    assert torch.equal(whole, before)
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
    nv.kv_append(cache, k[:0], k[:0], ints([], torch.int64))
    nv.kv_append(cache, k[:1], k[:1], ints([-1], torch.int64))
    assert torch.equal(whole, before) and nv.device_status() == 0


# ---- attention -------------------------------------------------------------------

def filled(nv, seqs, heads, dim, page, seed=0, layers=1, stale=255, blocks=None, dtype=FP32,
           gain=1.0):
    """A cache holding `seqs` tokens a request on scattered pages (all else 0xFF:
    NaN scales), and its block table (unused entries far outside the pool)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in seqs]
    pages = sum(need) + 3
    blocks = max(max(need, default=0), 1) + 2 if blocks is None else blocks
    kg, vg = ints([gain * 5 / 2688], FP32), ints([4.5 / 2688], FP32)
    cache, whole = make_cache(nv, pages, heads, dim, page, kg, vg, layers, layers - 1, fill=stale)
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    table = torch.full((len(seqs), blocks), 1 << 30, dtype=torch.int32)
    slots = []
    for r, (n, m) in enumerate(zip(seqs, need)):
        mine = [order.pop() for _ in range(m)]
        table[r, :m] = torch.tensor(mine, dtype=torch.int32)
        slots += [mine[i // page] * page + i % page for i in range(n)]
    total = len(slots)
    k = torch.randn((total, heads, dim), generator=gen, device="cuda") * gain
    v = torch.randn((total, heads, dim), generator=gen, device="cuda")
    nv.kv_append(cache, k.to(dtype), v.to(dtype), ints(slots, torch.int64))
    return cache, table.cuda(), gen


def starts(counts):
    return ints(list(itertools.accumulate(counts, initial=0)))


def run_attention(nv, seqs, counts, hq, hkv, dim, page, q_dtype=BF16, out_dtype=None, window=0,
                  scale=None, seed=0, layers=1, uniform=False, max_q="known", gain=1.0, **more):
    cache, table, gen = filled(nv, seqs, hkv, dim, page, seed, layers, gain=gain)
    rows = torch.randn((sum(counts), hq + 2 * hkv, dim), generator=gen, device="cuda").to(q_dtype)
    q = rows[:, :hq]
    nv.device_status(clear=True)
    out, lse = nv.kv_attention(cache, q, table, ints(seqs), None if uniform else starts(counts),
                               max_q=max(counts, default=0) if max_q == "known" else max_q, scale=scale,
                               window=window, out_dtype=out_dtype, return_lse=True, **more)
    assert nv.device_status() == 0
    assert out.dtype == (out_dtype or q_dtype)
    ref = attention(cache, q, table, seqs, counts, scale, window)
    check_attention(out, lse, ref, q_dtype)
    return cache, q, table, out, lse


@pytest.mark.parametrize("q_dtype,out_dtype", [(BF16, BF16), (FP32, FP32), (BF16, FP32), (FP32, BF16)])
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 64)])
def test_single_tokens(nv, q_dtype, out_dtype, dim, page):
    """One token a request, lengths around every boundary, an empty request."""
    seqs = [1, 0, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 1000]
    run_attention(nv, seqs, [1] * len(seqs), 8, 2, dim, page, q_dtype, out_dtype)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (7, 1), (8, 1), (9, 1), (16, 1), (34, 2),
                                    (40, 1), (64, 1), (32, 32)])
def test_head_groups(nv, hq, hkv):
    run_attention(nv, [77, 300], [1, 1], hq, hkv, 128, 32, seed=hq)
    run_attention(nv, [50], [1], hq, hkv, 64, 16, FP32, seed=hq)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_pages_and_layers(nv, page, dtype):
    run_attention(nv, [page * 3 - 1, page, page + 1, 5], [1, 2, 3, 4], 8, 4, 128, page, dtype, layers=3)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("counts", [[2, 1, 0, 5], [16, 9], [3, 40, 1], [130, 0, 33], [300]])
@pytest.mark.parametrize("past", [0, 1, 95])
def test_several_tokens(nv, dtype, dim, counts, past):
    """Drafted tokens, chunks and whole prompts: the causal edge inside tiles."""
    run_attention(nv, [c + past if c else 0 for c in counts], counts, 8, 2, dim, 16, dtype, seed=past)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 5000])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_window(nv, window, dtype):
    run_attention(nv, [400, 90, 1, 200], [1, 1, 1, 1], 8, 2, 128, 32, dtype, window=window)
    run_attention(nv, [400, 90, 7], [37, 90, 7], 8, 2, 64, 16, dtype, window=window)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_long(nv, dtype):
    """A request cut between many SMs, beside short ones and empty ones."""
    run_attention(nv, [20011, 0, 3, 4096, 0], [1] * 5, 8, 2, 128, 64, dtype)
    run_attention(nv, [9001, 10, 700], [5, 2, 1], 16, 2, 64, 16, dtype)


def test_many_requests(nv):
    rng = np.random.default_rng(5)
    seqs = rng.integers(0, 60, 700).tolist()
    run_attention(nv, seqs, [1] * 700, 4, 2, 64, 16)
    counts = [int(min(n, c)) for n, c in zip(seqs, rng.integers(0, 4, 700))]
    run_attention(nv, seqs, counts, 4, 2, 64, 16)


def test_more_rows_than_tokens(nv):
    """Rows at positions below 0 (and requests whose cache is empty) see nothing."""
    run_attention(nv, [3, 0, 20], [8, 4, 40], 8, 2, 64, 16)
    run_attention(nv, [3, 0, 20], [8, 4, 200], 8, 2, 128, 16, FP32)


def test_scale_and_hints(nv):
    for max_q in (0, 1, 1000, None):
        run_attention(nv, [60, 500], [20, 3], 8, 2, 128, 16, scale=0.3, max_q=max_q)
    run_attention(nv, [60, 500, 8], [4, 4, 4], 8, 2, 128, 16, FP32, scale=-0.1, uniform=True)
    run_attention(nv, [60, 500], [1, 1], 8, 2, 64, 16, scale=0.0)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_peaked_and_growing_scores(nv, dtype):
    """Scores of hundreds that keep rising along the request: the reference is raised many times."""
    cache, table, gen = filled(nv, [600, 600], 1, 64, 16, gain=1.0)
    q = torch.randn((2, 4, 64), generator=gen, device="cuda")
    k = torch.arange(600, device="cuda")[:, None, None] * (q[0, :1] / 100)
    k = torch.cat([k, k.flip(0)])
    v = torch.randn((1200, 1, 64), generator=gen, device="cuda")
    cache.k_g.copy_(nv.global_scale(k.contiguous()))
    slots = torch.cat([table[r, :38].long().repeat_interleave(16)[:600] * 16
                       + torch.arange(600, device="cuda") % 16 for r in range(2)])
    nv.kv_append(cache, k, v, slots)
    q = (q[:1] * 10).expand(2, 4, 64).contiguous().to(dtype)
    out, lse = nv.kv_attention(cache, q, table, ints([600, 600]), return_lse=True)
    check_attention(out, lse, attention(cache, q, table, [600, 600], [1, 1]), dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_query_magnitudes(nv, dtype):
    """Query rows of very large, very small, zero and mixed elements."""
    cache, table, gen = filled(nv, [100], 1, 128, 16)
    q = torch.randn((1, 6, 128), generator=gen, device="cuda")
    q[0, 0] *= 2.0 ** 90
    q[0, 1] *= 2.0 ** -90
    q[0, 2] = 0.0
    q[0, 3, ::2] *= 2.0 ** -12
    q[0, 4] *= 2.0 ** -126
    q = q.to(dtype)
    for scale, rows in ((2.0 ** -90, [0]), (2.0 ** 90, [1]), (0.1, [2, 3, 4, 5])):
        out, lse = nv.kv_attention(cache, q, table, ints([100]), scale=scale, return_lse=True)
        ref = attention(cache, q, table, [100], [1], scale)
        check_attention(out[:, rows], lse[:, rows], [x[:, rows] for x in ref], dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_nonfinite_query_stays_in_its_row(nv, dtype, bad):
    cache, table, gen = filled(nv, [40, 90], 2, 64, 16)
    q = torch.randn((4, 8, 64), generator=gen, device="cuda")
    clean = q.clone()
    q[2, 3, 7] = bad
    out, lse = nv.kv_attention(cache, q.to(dtype), table, ints([40, 90]), starts([1, 3]), return_lse=True)
    ref = attention(cache, clean.to(dtype), table, [40, 90], [1, 3])
    keep = torch.ones((4, 8), dtype=torch.bool, device="cuda")
    keep[2, 3] = False
    assert not torch.isfinite(out[2, 3]).any()
    check_attention(out[keep][None], lse[keep][None], [x[keep][None] for x in ref], dtype)


def test_zero_tensor_scales(nv):
    cache, table, gen = filled(nv, [50], 2, 128, 16)
    cache.k_g.zero_()
    q = torch.randn((1, 8, 128), generator=gen, device="cuda")
    out, lse = nv.kv_attention(cache, q, table, ints([50]), return_lse=True)
    check_attention(out, lse, attention(cache, q, table, [50], [1]), FP32)
    cache.v_g.zero_()
    assert not nv.kv_attention(cache, q, table, ints([50])).any()


@pytest.mark.parametrize("counts", [[1, 1, 1], [7, 1, 30], [200, 1, 150]])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_workspace_and_repeats(nv, counts, dtype):
    """The same bits every time; the workspace is zero again after each call as
    far as its counters go, can be shared by calls of any shape, and may be left out."""
    seqs = [9000, 300, 5000]
    ws = nv.kv_attention_workspace(128)
    cache, q, table, out, lse = run_attention(nv, seqs, counts, 8, 2, 128, 64, dtype, workspace=ws)
    for _ in range(3):
        o2, l2 = nv.kv_attention(cache, q, table, ints(seqs), starts(counts), max_q=max(counts),
                                 return_lse=True, workspace=ws)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        run_attention(nv, [3000, 5], [1, 1], 8, 2, 128, 64, dtype, workspace=ws)
    run_attention(nv, seqs, counts, 8, 2, 128, 64, dtype, workspace=False)
    run_attention(nv, seqs, counts, 8, 2, 128, 64, dtype, workspace=ws[:64])


def test_output_tensors_and_strides(nv):
    cache, table, gen = filled(nv, [70, 9], 2, 64, 16)
    q = torch.randn((2, 8, 64), generator=gen, device="cuda").to(BF16)
    want = nv.kv_attention(cache, q, table, ints([70, 9]))
    wide = torch.full((2, 20, 64), 7.0, dtype=BF16, device="cuda")
    got = nv.kv_attention(cache, q, table[:, :6], ints([70, 9]), out=wide[:, 4:12])
    assert torch.equal(got, want) and (wide[:, :4] == 7).all() and (wide[:, 12:] == 7).all()
    # rows that belong to no request are left alone
    out = torch.full((4, 8, 64), 7.0, dtype=BF16, device="cuda")
    nv.kv_attention(cache, torch.cat([q, q]), table, ints([70, 9]), ints([1, 2, 3]), max_q=1, out=out)
    assert (out[[0, 3]] == 7).all() and torch.equal(out[1], nv.kv_attention(
        cache, q[1:], table[:1], ints([70]))[0])


def test_bad_entries_are_reported(nv):
    """Page ids outside the pool (within the pages a request needs), lengths past the table."""
    cache, table, gen = filled(nv, [70, 40], 2, 64, 16)
    q = torch.randn((2, 8, 64), generator=gen, device="cuda")
    good = nv.kv_attention(cache, q, table, ints([70, 40]))
    for value in (-1, cache.num_pages, 1 << 30):
        broken = table.clone()
        broken[0, 2] = value
        nv.device_status(clear=True)
        out = nv.kv_attention(cache, q, broken, ints([70, 40]))
        assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
        assert torch.equal(out[1], good[1])
    nv.device_status(clear=True)
    nv.kv_attention(cache, q, table[:, :3], ints([70, 40]))
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
    nv.kv_attention(cache, q, table, ints([70, 40]), ints([-5, 1, 99]))
    nv.device_status(clear=True)


def test_offsets_past_32_bits(nv):
    """A pool of over 8 GB whose last pages are used."""
    page, heads, dim = 256, 8, 128
    pages = (9 << 30) // nv.kv_page_bytes(page, heads, dim)
    kg = ints([5 / 2688], FP32)
    cache, whole = make_cache(nv, pages, heads, dim, page, kg, kg, fill=0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((300, heads, dim), generator=gen, device="cuda")
    slots = torch.arange(300, device="cuda") + (pages - 2) * page
    nv.kv_append(cache, k, k, slots)
    table = ints([[pages - 2, pages - 1]])
    q = torch.randn((1, 32, dim), generator=gen, device="cuda").to(BF16)
    out, lse = nv.kv_attention(cache, q, table, ints([300]), return_lse=True)
    check_attention(out, lse, attention(cache, q, table, [300], [1]), BF16)
    kk, _ = page_values(cache.pool[-2:], page, dim)
    assert (kk[0].transpose(0, 1) * kg.double() - k[:256].double()).abs().max() < 1.0


def test_streams_and_graphs(nv):
    """A step on a side stream and in a captured graph gives the eager bits."""
    seqs, page = [100, 3000, 15], 16
    cache, table, gen = filled(nv, seqs, 2, 64, page, blocks=200)
    k = torch.randn((3, 2, 64), generator=gen, device="cuda").to(BF16)
    q = torch.randn((3, 8, 64), generator=gen, device="cuda").to(BF16)
    free = ints([cache.num_pages - 1 - i for i in range(3)])
    new, head = ints([1, 1, 1]), ints([0])

    def step(lens, pdl):
        t = nv.kv_tables(lens, new, free, head, table, page_size=page, tokens=3, pdl=pdl)
        nv.kv_append(cache, k, k, t.slots, pdl=pdl)
        return nv.kv_attention(cache, q, table, t.seq_len, t.q_start, max_q=1, pdl=pdl), t.seq_len

    lens = ints(seqs)
    want, seq = step(lens, False)
    want = want.clone()
    assert seq.tolist() == [101, 3001, 16]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = step(lens, True)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = step(lens, True)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert torch.equal(step(lens, False)[0], want)


# ---- the tcgen05 kernel by name ----------------------------------------------------

def run_tile(nv, seqs, counts, hq, hkv, dim, page, **more):
    return run_attention(nv, seqs, counts, hq, hkv, dim, page, kernel=nv.KERNEL_KV_TILE, **more)


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("n", [1, 16, 100, 128, 129, 300])
def test_tile_one_request(nv, dim, n):
    run_tile(nv, [n], [1], 4, 1, dim, 16, seed=n)
    run_tile(nv, [n], [n], 4, 1, dim, 16, seed=n)


@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16), (128, 256)])
@pytest.mark.parametrize("counts", [[2, 1, 0, 5], [16, 9], [64, 65, 1], [130, 0, 33], [300], [700, 3, 1, 90]])
@pytest.mark.parametrize("past", [0, 1, 95, 1000])
def test_tile_several_tokens(nv, dim, page, counts, past):
    run_tile(nv, [c + past if c else 0 for c in counts], counts, 8, 2, dim, page, seed=past)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (7, 1), (16, 1), (40, 1), (64, 1), (32, 32)])
def test_tile_head_groups(nv, hq, hkv):
    run_tile(nv, [77, 300, 41], [5, 70, 41], hq, hkv, 128, 32, seed=hq)


@pytest.mark.parametrize("window", [1, 2, 100, 127, 128, 129, 5000])
def test_tile_window(nv, window):
    run_tile(nv, [400, 90, 7, 1000], [37, 90, 7, 400], 8, 2, 128, 16, window=window)
    run_tile(nv, [1500], [1], 8, 2, 64, 16, window=window)


def test_tile_empty_and_early_rows(nv):
    run_tile(nv, [0, 3, 0, 20], [1, 8, 4, 200], 8, 2, 128, 16)
    run_tile(nv, [0, 0], [1, 1], 8, 2, 64, 16)


def test_tile_scale(nv):
    for scale in (0.3, -0.1, 0.0):
        run_tile(nv, [260, 500], [20, 3], 8, 2, 128, 16, scale=scale)


@pytest.mark.parametrize("counts", [[1, 1], [300, 1], [900, 40]])
def test_tile_workspace_and_repeats(nv, counts):
    """Items cut between many SMs; the same bits each time; no workspace: no cuts."""
    seqs = [9000, 3000]
    cache, q, table, out, lse = run_tile(nv, seqs, counts, 8, 2, 128, 64)
    for _ in range(3):
        o2, l2 = nv.kv_attention(cache, q, table, ints(seqs), starts(counts), return_lse=True,
                                 kernel=nv.KERNEL_KV_TILE)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        run_attention(nv, [3000, 5], [1, 1], 8, 2, 128, 64)
    run_tile(nv, seqs, counts, 8, 2, 128, 64, workspace=False)


def test_tile_nonfinite_query_stays_in_its_row(nv):
    cache, table, gen = filled(nv, [140, 290], 2, 64, 16)
    for bad in (math.nan, math.inf):
        q = torch.randn((103, 8, 64), generator=gen, device="cuda")
        clean = q.to(BF16)
        q[50, 3, 7] = bad
        out, lse = nv.kv_attention(cache, q.to(BF16), table, ints([140, 290]), starts([100, 3]),
                                   return_lse=True, kernel=nv.KERNEL_KV_TILE)
        ref = attention(cache, clean, table, [140, 290], [100, 3])
        keep = torch.ones((103, 8), dtype=torch.bool, device="cuda")
        keep[50, 3] = False
        assert not torch.isfinite(out[50, 3]).any()
        check_attention(out[keep][None], lse[keep][None], [x[keep][None] for x in ref], BF16)


def test_tile_zero_tensor_scale_and_bad_pages(nv):
    cache, table, gen = filled(nv, [200, 40], 2, 128, 16)
    q = torch.randn((60, 8, 128), generator=gen, device="cuda").to(BF16)
    args = (ints([200, 40]), starts([40, 20]))
    good = nv.kv_attention(cache, q, table, *args, kernel=nv.KERNEL_KV_TILE)
    broken = table.clone()
    broken[0, 2] = cache.num_pages
    nv.device_status(clear=True)
    out = nv.kv_attention(cache, q, broken, *args, kernel=nv.KERNEL_KV_TILE)
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
    assert torch.equal(out[40:], good[40:])
    cache.k_g.zero_()
    out, lse = nv.kv_attention(cache, q, table, *args, return_lse=True, kernel=nv.KERNEL_KV_TILE)
    check_attention(out, lse, attention(cache, q, table, [200, 40], [40, 20]), BF16)


def test_tile_wants_bf16(nv):
    cache, table, gen = filled(nv, [20], 1, 64, 16)
    q = torch.randn((2, 4, 64), generator=gen, device="cuda")
    for x, dtype in ((q, FP32), (q.to(BF16), FP32), (q, BF16)):
        with pytest.raises(nv.Nvfp4Error):
            nv.kv_attention(cache, x, table, ints([20]), out_dtype=dtype, kernel=nv.KERNEL_KV_TILE)


def test_growing_scores_in_tiles(nv):
    """Scores that rise along the keys: outputs are rescaled in tensor memory again and again."""
    cache, table, gen = filled(nv, [900], 1, 64, 16)
    base = torch.randn((64,), generator=gen, device="cuda")
    k = torch.arange(900, device="cuda")[:, None, None] * (base / 100)
    v = torch.randn((900, 1, 64), generator=gen, device="cuda")
    cache.k_g.copy_(nv.global_scale(k.contiguous()))
    slots = table[0, :57].long().repeat_interleave(16)[:900] * 16 + torch.arange(900, device="cuda") % 16
    nv.kv_append(cache, k.contiguous(), v, slots)
    q = (base * 10 + torch.randn((300, 4, 64), generator=gen, device="cuda")).to(BF16)
    for kernel in (nv.KERNEL_KV_ROWS, nv.KERNEL_KV_TILE):
        out, lse = nv.kv_attention(cache, q, table, ints([900]), return_lse=True, kernel=kernel)
        check_attention(out, lse, attention(cache, q, table, [900], [300]), BF16)


# ---- append, more ----------------------------------------------------------------------

def test_append_ties_and_signs(nv):
    """Elements on every rounding boundary of E2M1, both signs, zeros of both
    signs, saturation; the block scale is exactly 1 (maximum 6, tensor scale 1)."""
    grid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    vals = grid + [np.nextafter(np.float32(x), np.float32(s)) for x in grid[:7] for s in (0, 9)] + [0.0]
    x = torch.tensor(np.array(vals + [-v for v in vals], np.float32))
    rows = x[torch.randint(0, len(x), (64, 128), generator=torch.Generator().manual_seed(1))]
    rows[:, ::16] = 6.0
    rows[::2, 5::16] = -0.0
    rows = rows.cuda()
    one = ints([1.0], FP32)
    cache, whole = make_cache(nv, 4, 1, 128, 16, one, one)
    nv.kv_append(cache, rows[:, None], -rows[:, None], torch.arange(64, device="cuda"))
    kk, vv = page_values(cache.pool, 16, 128)
    for got, want in ((kk, rows), (vv, -rows)):
        q, s = oracle.quantize(want.cpu().numpy(), np.float32(1.0))
        q = torch.from_numpy(q).cuda()
        part = cache.pool[:, 0, :1024] if want is rows else cache.pool[:, 0, 1024:2048]
        assert torch.equal(part.reshape(64, 64), q)
        assert (s == 0x38).all()
        assert (got[:, 0].reshape(64, 128) - want.double()).abs().max() <= 1.0


@pytest.mark.parametrize("scale", [2.0 ** -130, 2.0 ** -110, 2.0 ** 105, 2.0 ** 118])
def test_append_extreme_magnitudes(nv, scale):
    """Blocks whose scale leaves the domain of the reciprocal's correction."""
    x = (torch.randn((40, 2, 64), generator=torch.Generator().manual_seed(3)) * scale).cuda()
    x[3] = 0.0
    g = nv.global_scale(x)
    cache, whole = make_cache(nv, 3, 2, 64, 16, g, g)
    nv.kv_append(cache, x, x, torch.arange(40, device="cuda"))
    q, s = oracle.quantize(x.cpu().numpy().reshape(80, 64), np.float32(g.item()))
    got = torch.cat([cache.pool[t // 16, h, t % 16 * 32:t % 16 * 32 + 32][None]
                     for t in range(40) for h in range(2)])
    assert torch.equal(got.cpu(), torch.from_numpy(q))


@pytest.mark.parametrize("tokens", [9000, 30001])
def test_append_many_tokens(nv, tokens):
    """Many tokens (several a thread), unaligned BF16 rows, against few at a time."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    flat = torch.randn((tokens, 2 * 4 * 64 + 4), generator=gen, device="cuda").to(BF16)
    k, v = (flat[:, 4 + 256 * i:4 + 256 * (i + 1)].unflatten(1, (4, 64)) for i in range(2))
    g = ints([0.002], FP32)
    pages = -(-tokens // 64) + 1
    a, pool_a = make_cache(nv, pages, 4, 64, 64, g, g, fill=0)
    b, pool_b = make_cache(nv, pages, 4, 64, 64, g, g, fill=0)
    slots = torch.randperm(pages * 64, generator=gen, device="cuda")[:tokens].contiguous()
    slots[5::11] = -1
    nv.kv_append(a, k, v, slots)
    for i in range(0, tokens, 1000):
        nv.kv_append(b, k[i:i + 1000].float().contiguous(), v[i:i + 1000].float().contiguous(), slots[i:i + 1000])
    assert torch.equal(pool_a, pool_b)


# ---- what the binding refuses ------------------------------------------------------------

def test_binding_refusals(nv):
    cache, table, gen = filled(nv, [20, 9], 2, 64, 16)
    q = torch.randn((2, 8, 64), generator=gen, device="cuda")
    lens = ints([20, 9])
    ok = dict(cache=cache, q=q, block_table=table, seq_len=lens)
    for change in (dict(q=q.half()), dict(q=q.cpu()), dict(q=q[0]), dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1)),
                   dict(q=q[:, :7]), dict(block_table=table.long()), dict(block_table=table[:1]),
                   dict(block_table=table.T), dict(seq_len=lens.long()), dict(seq_len=lens[:1].cpu()),
                   dict(q_start=lens), dict(q_start=ints([0, 1, 2], torch.int64)), dict(out=q[:1]),
                   dict(out=q.half()), dict(out_dtype=torch.float16), dict(q=torch.cat([q, q[:1]])),
                   dict(workspace=torch.zeros(100, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            nv.kv_attention(**{**ok, **change})
    for change in (dict(window=-1), dict(scale=math.nan), dict(kernel=77)):
        with pytest.raises(nv.Nvfp4Error):
            nv.kv_attention(**{**ok, **change})
    with pytest.raises(TypeError):
        nv.kv_attention(**{**ok, "scale": "x"})
    k = torch.randn((3, 2, 64), device="cuda")
    slots = torch.arange(3, device="cuda")
    for args in ((k, k[:2], slots), (k, k.to(BF16), slots), (k, k, slots.to(torch.int32)), (k, k, slots[:2]),
                 (k[:, :1], k[:, :1], slots), (k.transpose(0, 1), k, slots), (k.cpu(), k.cpu(), slots), (None, k, slots)):
        with pytest.raises(ValueError):
            nv.kv_append(cache, *args)
    t = dict(kv_len=lens, q_len=lens, free_pages=lens, free_head=lens[:1], block_table=table, page_size=16, tokens=29)
    for change in (dict(q_len=lens[:1]), dict(kv_len=lens.float()), dict(free_head=lens), dict(tokens=-1),
                   dict(block_table=table[:1]), dict(free_pages=lens.cpu()), dict(out=(lens,) * 5)):
        with pytest.raises(ValueError):
            nv.kv_tables(**{**t, **change})
    with pytest.raises(nv.Nvfp4Error):
        nv.kv_tables(**{**t, "page_size": 20})
    assert nv.device_status() == 0


def test_tables_into_given_tensors(nv):
    past, new, free = ints([5, 16]), ints([3, 1]), ints([7, 8, 9])
    table = ints([[1, -1], [2, -1]])
    first = nv.kv_tables(past, new, free, ints([0]), table, page_size=16, tokens=6)
    out = nv.KVTables(*(torch.full_like(x, 77) for x in first))
    again = nv.kv_tables(past, new, free, ints([0]), table, page_size=16, tokens=6, out=out)
    assert again is out
    for a, b in zip(first, out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("reqs,tokens", [(1, 1), (3, 0), (5, 7), (8, 33)])
def test_tables_outputs_are_separate(nv, reqs, tokens):
    past, new = ints([4] * reqs), ints([1] * reqs)
    table = torch.full((reqs, 2), 3, dtype=torch.int32, device="cuda")
    got = nv.kv_tables(past, new, ints([7]), ints([0]), table, page_size=16, tokens=max(tokens, reqs))
    sizes = [reqs, reqs + 1, max(tokens, reqs), max(tokens, reqs), 1]
    for i, (t, n) in enumerate(zip(got, sizes)):
        assert t.shape == (n,) and t.is_contiguous() and t.data_ptr() % 16 == 0
        assert t.dtype == (torch.int64 if i == 2 else torch.int32)
        t.fill_(-100 - i)                                  # each has its own bytes
    for i, t in enumerate(got):
        assert (t == -100 - i).all()
    kept = got.positions
    del got
    other = torch.zeros(1 << 12, dtype=torch.int32, device="cuda")  # takes freed memory, if there is any
    assert (kept == -103).all() and (other == 0).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shift,extra", [(4, 0), (0, 4), (4, 4)])
def test_rows_on_8_byte_boundaries(nv, dim, shift, extra):
    """BF16 queries and outputs that are aligned to 8 bytes only give what aligned copies give."""
    lens = [300, 41]
    cache, table, gen = filled(nv, lens, 2, dim, 32)
    row = 8 * dim + extra
    flat = torch.randn(80 * row + 8, generator=gen, device="cuda").to(BF16)
    q = flat[shift:].as_strided((80, 8, dim), (row, dim, 1))
    start = ints([0, 47, 80])
    for kernel in (nv.KERNEL_KV_ROWS, nv.KERNEL_KV_TILE):
        want = nv.kv_attention(cache, q.contiguous(), table, ints(lens), start, max_q=47, kernel=kernel)
        room = torch.full((80 * row + 8,), 7.0, dtype=BF16, device="cuda")
        out = room[shift:].as_strided((80, 8, dim), (row, dim, 1))
        nv.kv_attention(cache, q, table, ints(lens), start, max_q=47, kernel=kernel, out=out)
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert (room == 7.0).all()                      # nothing else was written


# ---- waits -------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_ring_of_groups_that_end_early(nv, dtype):
    """Groups of 64 tokens whose second half lies past the request's end (their warp gives
    the ring's place back unread), many of them in a row and in every share: no wait runs
    out and the bits repeat."""
    rng = np.random.default_rng(11)
    seqs = (64 * rng.integers(0, 12, 600) + rng.integers(1, 33, 600)).tolist()
    cache, q, table, out, lse = run_attention(nv, seqs, [1] * 600, 8, 2, 64, 16, dtype)
    for _ in range(20):
        o2, l2 = nv.kv_attention(cache, q, table, ints(seqs), starts([1] * 600), max_q=1, return_lse=True)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert nv.device_status() == 0


def test_tile_waits_of_whole_warps(nv):
    """Items of one and of two tiles in turn, cut and whole: every wait of the softmax
    warps before their loads of scores and outputs; the bits repeat and none runs out."""
    counts = [130, 3, 64, 300, 1, 33] * 4
    seqs = [c + 700 * (i % 3) for i, c in enumerate(counts)]
    cache, q, table, out, lse = run_tile(nv, seqs, counts, 8, 2, 64, 16)
    for _ in range(20):
        o2, l2 = nv.kv_attention(cache, q, table, ints(seqs), starts(counts), return_lse=True,
                                 kernel=nv.KERNEL_KV_TILE)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    assert nv.device_status() == 0


# ---- block tables at the largest lengths ------------------------------------------------------

BIG = 2 ** 31 - 1


@pytest.mark.parametrize("past,new,tokens", [
    ([BIG], [5], 8), ([BIG - 3, 4], [5, 2], 7), ([3, BIG, 7], [1, BIG, 2], 40), ([0, 3], [BIG, BIG], 40),
    ([0] * 4, [2 ** 30] * 4, 33), ([BIG] * 600, [BIG] * 600, 700), ([5, 0], [3, BIG], 90)])
def test_tables_lengths_up_to_int32(nv, past, new, tokens):
    """Positions and sums that pass 32 bits are cut off and reported; the table is never
    left (a guard of 64 rows on both sides of it stays as it was)."""
    page, blocks, reqs = 16, 4, len(past)
    cap = page * blocks
    free = list(range(100, 100 + 3 * reqs))
    room = torch.full((reqs + 128, blocks), -9, dtype=torch.int32, device="cuda")
    table = room[64:64 + reqs]
    held = [-(-min(n, cap) // page) for n in past]
    for r, h in enumerate(held):
        table[r, :h] = 10000 + r
    rows, seq, start, head, want = [], [], [0], 1, table.tolist()
    for r, (n, c) in enumerate(zip(past, new)):
        end = min(n + c, cap)
        for b in range(held[r], -(-end // page)):
            want[r][b] = free[head] if head < len(free) else -1
            head += 1
        for i in range(min(c, tokens - len(rows))):
            pos = n + i
            entry = want[r][pos // page] if pos < end else -1
            rows.append((min(pos, BIG), entry * page + pos % page if entry >= 0 else -1))
        seq.append(end)
        start.append(start[-1] + c)
    rows += [(0, -1)] * (tokens - len(rows))
    nv.device_status(clear=True)
    got = nv.kv_tables(ints(past), ints(new), ints(free), ints([1]), table, page_size=page, tokens=tokens)
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
    assert got.seq_len.tolist() == seq
    assert got.q_start.tolist() == [min(s, BIG) for s in start]
    assert got.positions.tolist() == [p for p, _ in rows]
    assert got.slots.tolist() == [s for _, s in rows]
    assert got.free_head.tolist() == [head]
    assert table.tolist() == want
    assert (room[:64] == -9).all() and (room[64 + reqs:] == -9).all()


def test_tables_pages_past_32_bits(nv):
    """More than 2^32 new pages in a table of 17 GB: those past the free list are -1, all of them."""
    reqs, blocks = 16384, (1 << 18) + 1
    table = torch.full((reqs, blocks), 7, dtype=torch.int32, device="cuda")
    new = torch.full((reqs,), BIG, dtype=torch.int32, device="cuda")
    nv.device_status(clear=True)
    got = nv.kv_tables(torch.zeros_like(new), new, ints([50, 51, 52]), ints([-2]), table, page_size=16, tokens=100)
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
    assert table[0, :6].tolist() == [-1, -1, 50, 51, 52, -1]
    table[0, 2:5] = -1
    for rows in table.split(1024):
        assert (rows == -1).all()
    assert got.free_head.tolist() == [BIG] and got.q_start[-1].item() == BIG
    assert got.slots[:32].tolist() == [-1] * 32 and got.slots[32:80].tolist() == list(range(800, 848))


# ---- pages that are not there ---------------------------------------------------------------

def without_pages(nv, cache, pages):
    """The same cache with these pages' bytes zero."""
    pool = cache.pool.clone()
    pool[pages] = 0
    return nv.KVCache(pool, cache.k_g, cache.v_g, page_size=cache.page_size, head_dim=cache.head_dim)


@pytest.mark.parametrize("name,dtype", [("KERNEL_KV_ROWS", BF16), ("KERNEL_KV_ROWS", FP32), ("KERNEL_KV_TILE", BF16)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_pages_outside_the_pool_count_as_zeros(nv, name, dtype, page):
    """Not as what an earlier request left in the place that a page is copied to."""
    kernel = getattr(nv, name)
    seqs, counts = [900, 40], [3, 2]
    other, other_table, _ = filled(nv, [20000] * 8, 2, 64, 64, seed=9)
    cache, table, gen = filled(nv, seqs, 2, 64, page)
    q = torch.randn((5, 8, 64), generator=gen, device="cuda").to(dtype)
    for at in ([0], [2, 3], [-(-900 // page) - 1], list(range(-(-900 // page)))):
        lost = table[0, at].long()
        ref = attention(without_pages(nv, cache, lost), q, table, seqs, counts)
        for value in (-1, cache.num_pages, 1 << 30):
            broken = table.clone()
            broken[0, at] = value
            # what the SMs' shared memory holds before: keys and values of other requests
            nv.kv_attention(other, q.repeat(2, 1, 1)[:8], other_table, ints([20000] * 8), kernel=kernel)
            nv.device_status(clear=True)
            out, lse = nv.kv_attention(cache, q, broken, ints(seqs), starts(counts), max_q=3, return_lse=True,
                                       kernel=kernel)
            assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
            check_attention(out, lse, ref, dtype)


@pytest.mark.parametrize("name,dtype", [("KERNEL_KV_ROWS", BF16), ("KERNEL_KV_ROWS", FP32), ("KERNEL_KV_TILE", BF16)])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (64, 64), (128, 128), (64, 256)])
@pytest.mark.parametrize("window", [1, 37, 100, 256])
def test_pages_that_a_window_has_left(nv, name, dtype, dim, page, window):
    """Keys before every row's window: NaN bytes, or pages given away and their entries gone."""
    kernel = getattr(nv, name)
    seqs, counts = [1000, 400, 90, 777], [1, 5, 90, 40]
    cache, table, gen = filled(nv, seqs, 2, dim, page)
    q = torch.randn((sum(counts), 8, dim), generator=gen, device="cuda").to(dtype)
    args = dict(max_q=max(counts), window=window, return_lse=True, kernel=kernel)
    good, good_lse = nv.kv_attention(cache, q, table, ints(seqs), starts(counts), **args)
    check_attention(good, good_lse, attention(cache, q, table, seqs, counts, window=window), dtype)
    half, block = page * dim // 2, page * dim // 16
    parts = [cache.pool[:, :, a:a + page * n].unflatten(2, (page, n)) for a, n in (
        (0, dim // 2), (half, dim // 2), (2 * half, dim // 16), (2 * half + block, dim // 16))]
    firsts = [max(0, n - c - window + 1) for n, c in zip(seqs, counts)]
    for r, first in enumerate(firsts):
        pos = torch.arange(first, device="cuda")
        for part in parts:
            part[table[r, pos // page].long(), :, pos % page] = 255
    for entry in (None, -1, cache.num_pages):
        left = table.clone()
        for r, first in enumerate(firsts):
            if entry is not None:
                left[r, :first // page] = entry
        nv.device_status(clear=True)
        out, lse = nv.kv_attention(cache, q, left, ints(seqs), starts(counts), **args)
        assert nv.device_status(clear=True) == 0
        assert torch.equal(out, good) and torch.equal(lse, good_lse)


@pytest.mark.parametrize("name", ["KERNEL_KV_ROWS", "KERNEL_KV_TILE"])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_every_entry_below_zero_is_reported(nv, name, page):
    cache, table, gen = filled(nv, [300, 40], 2, 64, page)
    q = torch.randn((2, 8, 64), generator=gen, device="cuda").to(BF16)
    ref = attention(without_pages(nv, cache, table[0, 1:2].long()), q, table, [300, 40], [1, 1])
    for value in (-1, -2, -3, -77, -2 ** 31):
        broken = table.clone()
        broken[0, 1] = value
        nv.device_status(clear=True)
        out, lse = nv.kv_attention(cache, q, broken, ints([300, 40]), return_lse=True, kernel=getattr(nv, name))
        assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
        check_attention(out, lse, ref, BF16)


# ---- rows of no request ----------------------------------------------------------------------

@pytest.mark.parametrize("name,q_dtype,out_dtype", [("KERNEL_KV_ROWS", BF16, BF16), ("KERNEL_KV_ROWS", FP32, FP32),
                                                    ("KERNEL_KV_ROWS", BF16, FP32), ("KERNEL_KV_TILE", BF16, BF16)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("counts,before,after", [([1, 1, 1], 0, 5), ([1, 1, 1], 2, 0), ([60, 0, 3], 3, 700),
                                                 ([0, 0, 0], 0, 9), ([0, 0, 0], 6, 0), ([], 0, 7), ([], 3, 1)])
def test_rows_of_no_request(nv, name, q_dtype, out_dtype, dim, counts, before, after):
    """Zeros and -inf in new outputs, whatever their memory held; given outputs keep them."""
    kernel = getattr(nv, name)
    seqs = [300 + c for c in counts]
    cache, table, gen = filled(nv, seqs or [5], 2, dim, 16)
    table = table[:len(counts)]
    tokens = before + sum(counts) + after
    q = torch.randn((tokens, 14, dim), generator=gen, device="cuda").to(q_dtype)
    start = ints([before + s for s in itertools.accumulate(counts, initial=0)])
    mine = slice(before, before + sum(counts))
    ref = attention(cache, q[mine], table, seqs, counts)
    args = dict(max_q=max(counts, default=0), out_dtype=out_dtype, kernel=kernel)
    lens = ints(seqs)
    for _ in range(3):
        # the call takes memory that held this
        old = [torch.full((tokens, 14, dim), math.nan, dtype=out_dtype, device="cuda") for _ in range(8)]
        old += [torch.full((tokens, 14), math.nan, device="cuda") for _ in range(8)]
        del old
        out, lse = nv.kv_attention(cache, q, table, lens, start, return_lse=True, **args)
        if sum(counts):
            check_attention(out[mine], lse[mine], ref, q_dtype)
        for rows in (slice(0, before), slice(before + sum(counts), tokens)):
            assert not out[rows].any() and (lse[rows] == -math.inf).all()
    given = torch.full((tokens, 16, dim), 7.0, dtype=out_dtype, device="cuda")
    got, lse2 = nv.kv_attention(cache, q, table, lens, start, out=given[:, 1:15], return_lse=True, **args)
    assert torch.equal(got[mine], out[mine]) and torch.equal(lse2, lse)
    given[mine, 1:15] = 7.0
    assert (given == 7.0).all()


def test_rows_without_requests_or_starts(nv):
    cache, table, gen = filled(nv, [5], 2, 64, 16)
    q = torch.randn((6, 4, 64), generator=gen, device="cuda")
    none = ints([])
    out, lse = nv.kv_attention(cache, q, table[:0], none, return_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    assert nv.kv_attention(cache, q[:0], table[:0], none).shape == (0, 4, 64)


def test_padded_step_into_a_linear(nv):
    """Tables, append, attention and the o linear of a step of 8 rows with 5 requests."""
    page, reqs, tokens, hq, hkv, dim = 16, 5, 8, 8, 2, 64
    cache, table, gen = filled(nv, [40, 3, 17, 100, 9], hkv, dim, page)
    lens = [40, 3, 17, 100, 9]
    free = ints([cache.num_pages - 1 - i for i in range(3)])
    for r, n in enumerate(lens):
        table[r, -(-n // page):] = -1
    w = nv.pack_weight(torch.randn((128, hq * dim), generator=gen, device="cuda"))
    rows = torch.randn((tokens, hq + 2 * hkv, dim), generator=gen, device="cuda").to(BF16)
    t = nv.kv_tables(ints(lens), ints([1] * reqs), free, ints([0]), table, page_size=page, tokens=tokens)
    nv.kv_append(cache, rows[:, hq:hq + hkv], rows[:, hq + hkv:], t.slots)
    bad = torch.full((tokens, hq, dim), math.nan, dtype=BF16, device="cuda")
    del bad
    y = nv.kv_attention(cache, rows[:, :hq], table, t.seq_len, t.q_start, max_q=1)
    z = nv.linear(y.flatten(1), cache.v_g, *w)
    assert torch.isfinite(z).all() and not z[reqs:].any() and z[:reqs].any(1).all()


# ---- probabilities of a block whose second half raises the reference --------------------------

@pytest.mark.parametrize("name", ["KERNEL_KV_ROWS", "KERNEL_KV_TILE"])
def test_probabilities_are_rounded_once(nv, name):
    """One f16 rounding of each probability (the bound's 2^-11), also where the reference rises
    inside a block: 128 keys of score 0, 64 about 2^7 times as probable with values of +1, then 16
    about 2^9 times with values of -1, so that the rest of the two sums is what roundings leave."""
    n, group, tail = 256 + 64, 64, 64
    unit = 1.4426950408889634  # scores below are in powers of two
    cache, table, gen = filled(nv, [n], 1, 64, 16)
    k = torch.zeros((n, 1, 64), device="cuda")
    k[128:192, 0, 0] = 6.0
    k[192:208, 0, 16] = 6.0
    k[128:192, 0, 1] = k[192:208, 0, 17] = 0.5  # a twelfth, for scores between those of BF16 queries
    k[208:, 0, 32] = -6.0                     # as good as unseen
    v = torch.zeros((n, 1, 64), device="cuda")
    v[128:192], v[192:208] = 1.0, -1.0
    cache.k_g.fill_(1.0)
    cache.v_g.fill_(1.0)
    slots = table[0, :n // 16].long().repeat_interleave(16) * 16 + torch.arange(n, device="cuda") % 16
    nv.kv_append(cache, k, v, slots)
    q = torch.zeros((tail, group, 64), device="cuda")
    rand = lambda: torch.rand((tail, group), generator=gen, device="cuda")  # noqa: E731
    q[..., 1], q[..., 17] = rand(), rand()
    q[..., 0] = (7.0 + 0.08 * rand() - 0.5 * q[..., 1]) / 6.0
    q[..., 16] = (8.93 + 0.069 * rand() - 0.5 * q[..., 17]) / 6.0
    q[..., 32] = 10.0
    q = q.to(BF16)
    # (no workspace: a request's keys stay with one SM, in order)
    out, lse = nv.kv_attention(cache, q, table, ints([n]), scale=1.0 / unit, return_lse=True,
                               kernel=getattr(nv, name), workspace=False)
    check_attention(out, lse, attention(cache, q, table, [n], [tail], 1.0 / unit), BF16)


# ---- workspaces -------------------------------------------------------------------------------

@pytest.mark.parametrize("name,dtype,counts", [("KERNEL_KV_ROWS", BF16, [1, 1, 1]), ("KERNEL_KV_ROWS", FP32, [7, 1, 30]),
                                               ("KERNEL_KV_TILE", BF16, [200, 1, 150])])
def test_workspace_holds_anything_but_counters(nv, name, dtype, counts):
    """A new workspace has its counters zeroed and nothing else written: a graph that makes
    its own replays no fill of 40 MB.  What the rest held does not matter."""
    seqs, kernel = [9000, 300, 5000], getattr(nv, name)
    cache, q, table, out, lse = run_attention(nv, seqs, counts, 8, 2, 128, 64, dtype, kernel=kernel)
    zero = torch.zeros_like(nv.kv_attention_workspace(128))
    old = [torch.full_like(zero, 255) for _ in range(3)]           # NaN in FP32
    del old
    ws = nv.kv_attention_workspace(128)
    assert not ws[:4096].any() and (ws[4096:] == 255).all()
    for w in (ws, zero, ws):
        o2, l2 = nv.kv_attention(cache, q, table, ints(seqs), starts(counts), max_q=max(counts), return_lse=True,
                                 workspace=w, kernel=kernel)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        assert not w[:4096].any()


def test_graph_with_a_workspace_of_its_own(nv):
    """A default capture (its stream has no workspace yet), replayed beside eager calls."""
    seqs, counts = [9000, 300, 5000], [1, 1, 1]
    cache, q, table, out, lse = run_attention(nv, seqs, counts, 8, 2, 128, 64)
    lens, start = ints(seqs), starts(counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, got_lse = nv.kv_attention(cache, q, table, lens, start, max_q=1, return_lse=True)
        again, _ = nv.kv_attention(cache, q, table, lens, start, max_q=1, return_lse=True)
    for _ in range(4):
        for x in (got, got_lse, again):
            x.fill_(math.nan)
        graph.replay()
        eager = nv.kv_attention(cache, q, table, lens, start, max_q=1)
        for x in (got, again, eager):
            assert torch.equal(x, out)
        assert torch.equal(got_lse, lse)
