"""Attention behind shared prefixes and cross attention over the paged NVFP4 cache, through
the public entry points, against their definitions in 64 bits."""
import itertools
import math

import numpy as np
import pytest
import torch

import oracle
from kv_helpers import check_attention, page_values
from kv_rows_helpers import attend, rotated, shared_keys, table_values

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
KERNELS = [("KERNEL_AUTO", BF16), ("KERNEL_AUTO", FP32), ("KERNEL_KV_ROWS", BF16), ("KERNEL_KV_TILE", BF16)]


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


def starts(counts):
    return list(itertools.accumulate(counts, initial=0))


def make(nv, spans, heads, dim, page, seed=0, layers=1, gain=1.0, spare=3):
    """A cache that holds the tokens [lo, hi) of every span on pages of its own, all else 0xFF (NaN
    scales), and the spans' block tables, int32 on the CPU, entries without a page far outside the pool."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    need = [max(0, -(-hi // page) - lo // page) if hi > lo else 0 for lo, hi in spans]
    pages = sum(need) + spare
    whole = nv.kv_pool(pages * layers, heads, dim, page)
    whole.fill_(255)
    cache = nv.KVCache(whole.view(pages, layers, heads, -1)[:, layers - 1], ints([gain * 5 / 2688], FP32),
                       ints([4.5 / 2688], FP32), page_size=page, head_dim=dim)
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    blocks = max([-(-hi // page) for _, hi in spans] + [1]) + 2
    table = torch.full((len(spans), blocks), 1 << 30, dtype=torch.int32)
    slots = []
    for r, ((lo, hi), n) in enumerate(zip(spans, need)):
        for b in range(n):
            table[r, lo // page + b] = order.pop()
        slots += [table[r, i // page].item() * page + i % page for i in range(lo, hi)]
    k = torch.randn((len(slots), heads, dim), generator=gen, device="cuda") * gain
    v = torch.randn((len(slots), heads, dim), generator=gen, device="cuda")
    nv.kv_append(cache, k, v, ints(slots, torch.int64))
    return cache, table, gen


class Shared:
    """A call's operands: groups of (prefix, [(tokens behind it, rows of them)]); a request's first number
    is None for an empty one, and (n,) for one of n tokens in all that is read on its own pages."""

    def __init__(self, nv, groups, hq, hkv, dim, page, q_dtype, seed=0, layers=1, gain=1.0, before=(), after=()):
        spans, seqs, counts, sizes = [], [], [], []
        free = list(before), list(after)
        for prefix, reqs in [(0, free[0])] * bool(free[0]) + list(groups) + [(0, free[1])] * bool(free[1]):
            for own, rows in reqs:
                if own is None:
                    n, low = 0, 0
                elif isinstance(own, tuple):
                    n, low = own[0], 0
                else:
                    n, low = prefix + own, prefix
                spans.append((low, n))
                seqs.append(n)
                counts.append(rows)
        sizes = [len(reqs) for _, reqs in groups]
        self.prefix = [p for p, _ in groups]
        self.start = [len(free[0]) + s for s in starts(sizes)]
        both = [(0, p) for p in self.prefix] + spans
        self.cache, table, gen = make(nv, both, hkv, dim, page, seed, layers, gain)
        self.prefix_table, self.table = table[:len(groups)].cuda(), table[len(groups):].cuda()
        self.seqs, self.counts = seqs, counts
        rows = torch.randn((sum(counts), hq + 2 * hkv, dim), generator=gen, device="cuda").to(q_dtype)
        self.q, self.gen = rows[:, :hq], gen
        self.args = dict(prefix_table=self.prefix_table, block_table=self.table, group_start=ints(self.start),
                         max_q=max(counts, default=0), return_lse=True, prefix_len=ints(self.prefix),
                         seq_len=ints(seqs), q_start=ints(starts(counts)))

    def ref(self, scale=None, cache=None, q=None):
        cache = cache or self.cache
        keys = shared_keys(cache, self.prefix_table, self.prefix, self.start, self.table, self.seqs, self.counts)
        return attend(self.q if q is None else q, keys, self.counts, scale)

    def call(self, nv, q=None, **more):
        return nv.kv_attention_shared(self.cache, self.q if q is None else q, **{**self.args, **more})


def run_shared(nv, groups, hq=8, hkv=2, dim=64, page=16, q_dtype=BF16, scale=None, kernel="KERNEL_AUTO",
               out_dtype=None, call=(), **more):
    s = Shared(nv, groups, hq, hkv, dim, page, q_dtype, **more)
    nv.device_status(clear=True)
    out, lse = s.call(nv, scale=scale, kernel=getattr(nv, kernel), out_dtype=out_dtype, **dict(call))
    assert nv.device_status() == 0
    assert out.dtype == (out_dtype or q_dtype)
    check_attention(out, lse, s.ref(scale), q_dtype)
    return s, out, lse


PREFIXES = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 1000]


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 64), (64, 256)])
@pytest.mark.parametrize("prefix", PREFIXES)
def test_one_group_of_single_tokens(nv, kernel, dtype, dim, page, prefix):
    """Prefixes and own keys that end around every boundary, inside pages and at their ends."""
    run_shared(nv, [(prefix, [(n, 1) for n in (1, 2, 15, 16, 17, 64, 100, 129)])], 8, 2, dim, page, dtype,
               kernel=kernel, seed=prefix)


@pytest.mark.parametrize("q_dtype,out_dtype", [(BF16, FP32), (FP32, BF16)])
@pytest.mark.parametrize("dim", [64, 128])
def test_mixed_types(nv, q_dtype, out_dtype, dim):
    run_shared(nv, [(100, [(5, 1), (70, 3)]), (33, [(40, 30)])], 8, 2, dim, 16, q_dtype, out_dtype=out_dtype)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (7, 1), (9, 1), (16, 1), (34, 2), (64, 1), (32, 32)])
def test_head_groups(nv, kernel, dtype, hq, hkv):
    run_shared(nv, [(77, [(5, 1), (130, 2), (1, 1)])], hq, hkv, 128, 32, dtype, kernel=kernel, seed=hq)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("hq,hkv", [(7, 1), (5, 1), (1, 1), (9, 3)])
@pytest.mark.parametrize("dim", [64, 128])
def test_odd_numbers_of_rows(nv, kernel, dtype, hq, hkv, dim):
    """Rows times heads of every remainder, cut items and whole ones: what the passes leave each other
    lies on its boundaries."""
    for counts in ([1], [1, 1], [2, 1], [1, 1, 2], [3, 2], [5, 6]):
        run_shared(nv, [(300, [(9 + c, c) for c in counts])], hq, hkv, dim, 16, dtype, kernel=kernel)
    run_shared(nv, [(20000, [(9, 5), (700, 6)])], hq, hkv, dim, 64, dtype, kernel=kernel)


GROUPS = [
    # groups of different sizes, one empty, one without a prefix
    [(300, [(5, 1), (40, 1)]), (0, [(7, 1), (100, 2)]), (50, []), (16, [(1, 1)]), (129, [(3, 2), (20, 20), (64, 1)])],
    # empty requests first, between and last; requests without rows
    [(100, [(None, 1), (5, 1), (None, 3)]), (40, [(9, 0), (9, 1), (None, 0)])],
    # rows inside the prefix: a request inside it as a whole, and one that ends just behind it
    [(100, [((40,), 1), (5, 1), ((103,), 5), ((100,), 1), (1, 1)])],
    # more rows than tokens
    [(10, [((4,), 9), (3, 2)])],
    # a prefix that nobody is left with
    [(500, []), (20, [(4, 4)])],
]


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
def test_groups(nv, kernel, dtype, groups, dim, page):
    run_shared(nv, groups, 8, 2, dim, page, dtype, kernel=kernel)
    # and requests of no group on both sides
    run_shared(nv, groups, 8, 2, dim, page, dtype, kernel=kernel, before=[(30, 1), (None, 2)], after=[(200, 3)])


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("counts", [[2, 1, 5], [16, 9], [64, 65, 1], [130, 33], [300], [200, 3, 1, 90]])
@pytest.mark.parametrize("prefix,past", [(1, 0), (95, 0), (128, 1), (1000, 100)])
def test_several_tokens(nv, kernel, dtype, counts, prefix, past):
    """Drafted tokens, chunks and prompts behind a prefix: all rows of a group in one product."""
    run_shared(nv, [(prefix, [(c + past, c) for c in counts])], 8, 2, 128, 16, dtype, kernel=kernel, seed=past)
    run_shared(nv, [(prefix, [(c + past, c) for c in counts]), (77, [(c, c) for c in counts])], 4, 1, 64, 64, dtype,
               kernel=kernel, seed=past)


def test_the_choice_of_kernels(nv):
    """Prefixes by the tcgen05 kernel with own keys by the other, and the other way round."""
    run_shared(nv, [(2000, [(20 + i, 1) for i in range(90)])], 32, 8, 128, 64)        # many rows in all, few each
    run_shared(nv, [(100 + i, [(300, 40)]) for i in range(20)], 32, 8, 64, 16)        # several rows each, few groups' share
    run_shared(nv, [(100, [(300, 290), (5, 1)])], 32, 8, 64, 16)
    # hints that do not fit
    for max_q in (0, 1, 1000, None):
        run_shared(nv, [(60, [(20, 20), (500, 3)])], 8, 2, 128, 16, call=dict(max_q=max_q))


def test_long_prefixes(nv):
    run_shared(nv, [(20011, [(5, 1), (4096, 1), (1, 1)])], 8, 2, 128, 64)
    run_shared(nv, [(9001, [(10, 5), (700, 2)]), (15000, [(1, 1)])], 16, 2, 64, 16, FP32)


def test_many_requests_and_groups(nv):
    rng = np.random.default_rng(5)
    groups = [(int(rng.integers(0, 90)), [(int(n) or None, 1) for n in rng.integers(0, 40, rng.integers(0, 6))])
              for _ in range(200)]
    run_shared(nv, groups, 4, 2, 64, 16)
    run_shared(nv, groups, 4, 2, 64, 16, FP32)


def test_scales(nv):
    for kernel, dtype in KERNELS:
        for scale in (0.3, -0.1, 0.0):
            run_shared(nv, [(60, [(5, 1), (50, 9)])], 8, 2, 128, 16, dtype, scale=scale, kernel=kernel)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_scores_far_apart(nv, kernel, dtype):
    """Prefix scores hundreds above the own ones, hundreds below, and both large: the join."""
    for high in (True, False):
        s = Shared(nv, [(70, [(9, 1), (40, 3)])], 4, 1, 64, 16, dtype)
        q = s.q.float().abs() * 20
        k = torch.ones((70, 1, 64), device="cuda") * (3.0 if high else -3.0)
        row = s.prefix_table[0].long()
        slots = torch.tensor([row[i // 16] * 16 + i % 16 for i in range(70)], device="cuda")
        nv.kv_append(s.cache, k, torch.randn((70, 1, 64), generator=s.gen, device="cuda"), slots)
        q = q.to(dtype)
        out, lse = s.call(nv, q, kernel=getattr(nv, kernel), scale=0.25)
        check_attention(out, lse, s.ref(0.25, q=q), dtype)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_without_groups_and_without_starts(nv, kernel, dtype):
    """group_start None: one group of all; q_start None: the same rows each; no groups: no sharing."""
    s = Shared(nv, [(100, [(5, 2), (40, 2), (130, 2)])], 8, 2, 64, 16, dtype)
    args = dict(kernel=getattr(nv, kernel))
    want, want_lse = s.call(nv, **args)
    check_attention(want, want_lse, s.ref(), dtype)
    for more in (dict(group_start=None), dict(q_start=None), dict(group_start=None, q_start=None)):
        out, lse = s.call(nv, **args, **more)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    t = Shared(nv, [(96, [(9, 1), (40, 1)])], 8, 2, 64, 16, dtype)
    whole = t.table.clone()
    whole[:, :6] = t.prefix_table[0, :6]
    none = dict(prefix_table=t.prefix_table[:0], prefix_len=ints([]), group_start=ints([0]), block_table=whole)
    alone, alone_lse = t.call(nv, **args, **none)
    same, same_lse = nv.kv_attention(t.cache, t.q, whole, ints(t.seqs), ints([0, 1, 2]), max_q=1, return_lse=True, **args)
    assert torch.equal(alone, same) and torch.equal(alone_lse, same_lse)
    check_attention(alone, alone_lse, t.ref(), dtype)
    shared, shared_lse = t.call(nv, **args, block_table=whole)
    check_attention(shared, shared_lse, t.ref(), dtype)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("counts", [[1, 1, 1], [40, 1, 150]])
def test_repeats_workspaces_and_scratch(nv, kernel, dtype, counts):
    """The same bits each time, whatever the memory that calls take held before; no workspace: no cuts."""
    s, out, lse = run_shared(nv, [(9000, [(300 + c, c) for c in counts]), (3000, [(20, 1)])], 8, 2, 128, 64, dtype,
                             kernel=kernel)
    ws = nv.kv_attention_workspace(128)
    for i in range(4):
        old = [torch.full((1 << 20,), math.nan, device="cuda") for _ in range(6)]
        del old
        o2, l2 = s.call(nv, kernel=getattr(nv, kernel), workspace=ws if i % 2 else None)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        assert not ws[:4096].any()
    for none in (False, ws[:64]):
        o2, l2 = s.call(nv, kernel=getattr(nv, kernel), workspace=none)
        check_attention(o2, l2, s.ref(), dtype)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_given_outputs_and_rows_of_no_request(nv, kernel, dtype):
    s, out, lse = run_shared(nv, [(100, [(5, 1), (70, 40)]), (30, [(4, 2)])], 8, 2, 64, 16, dtype, kernel=kernel)
    tokens = sum(s.counts)
    q = torch.full((tokens + 9, 8, 64), math.nan, dtype=dtype, device="cuda")
    q[4:4 + tokens] = s.q
    start = ints([4 + x for x in starts(s.counts)])
    old = [torch.full((tokens + 9, 8, 64), math.nan, dtype=dtype, device="cuda") for _ in range(4)]
    del old
    got, got_lse = s.call(nv, q, q_start=start, kernel=getattr(nv, kernel))
    assert torch.equal(got[4:4 + tokens], out) and torch.equal(got_lse[4:4 + tokens], lse)
    for rows in (slice(0, 4), slice(4 + tokens, None)):
        assert not got[rows].any() and (got_lse[rows] == -math.inf).all()
    room = torch.full((tokens + 9, 12, 64), 7.0, dtype=dtype, device="cuda")
    got, got_lse = s.call(nv, q, q_start=start, kernel=getattr(nv, kernel), out=room[:, 2:10])
    assert torch.equal(got[4:4 + tokens], out) and torch.equal(got_lse[4:4 + tokens], lse)
    room[4:4 + tokens, 2:10] = 7.0
    assert (room == 7.0).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shift,extra", [(4, 0), (0, 4), (4, 4)])
def test_rows_on_8_byte_boundaries(nv, dim, shift, extra):
    s = Shared(nv, [(200, [(90, 47), (41, 33)])], 8, 2, dim, 32, BF16)
    row = 8 * dim + extra
    flat = torch.zeros(80 * row + 8, dtype=BF16, device="cuda")
    q = flat[shift:].as_strided((80, 8, dim), (row, dim, 1))
    q.copy_(s.q)
    for kernel in (nv.KERNEL_KV_ROWS, nv.KERNEL_KV_TILE):
        want, _ = s.call(nv, kernel=kernel)
        room = torch.full((80 * row + 8,), 7.0, dtype=BF16, device="cuda")
        out = room[shift:].as_strided((80, 8, dim), (row, dim, 1))
        s.call(nv, q, kernel=kernel, out=out)
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert (room == 7.0).all()


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("page", [16, 64, 128])
def test_pages_outside_the_pool(nv, kernel, dtype, page):
    """Of the prefix and of a request: their keys count as zeros, reported; the rest is right."""
    s = Shared(nv, [(300, [(5, 1), (200, 3)]), (40, [(9, 2)])], 8, 2, 64, page, dtype)
    for which, at in (("prefix_table", (0, 1)), ("table", (1, -(-500 // page) - 1))):
        tables = dict(prefix_table=s.prefix_table, block_table=s.table)
        name = "block_table" if which == "table" else which
        pool = s.cache.pool.clone()
        pool[tables[name][at].long()] = 0
        zeroed = nv.KVCache(pool, s.cache.k_g, s.cache.v_g, page_size=page, head_dim=64)
        ref = s.ref(cache=zeroed)
        for value in (-1, -2, s.cache.num_pages, 1 << 30):
            broken = tables[name].clone()
            broken[at] = value
            nv.device_status(clear=True)
            out, lse = s.call(nv, kernel=getattr(nv, kernel), **{name: broken})
            assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
            check_attention(out, lse, ref, dtype)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_lengths_past_the_tables(nv, kernel, dtype):
    """A prefix past its table is cut off there and reported; other groups are right.  Bad
    starts and groups lead nowhere outside (their results mean nothing)."""
    s = Shared(nv, [(300, [(5, 1), (200, 3)]), (40, [(9, 2)])], 8, 2, 64, 16, dtype)
    args = dict(kernel=getattr(nv, kernel))
    want, _ = s.call(nv, **args)
    nv.device_status(clear=True)
    out, _ = s.call(nv, **args, prefix_table=s.prefix_table[:, :10].contiguous())
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
    assert torch.equal(out[4:], want[4:])
    for more in (dict(prefix_len=ints([2 ** 31 - 1, -5])), dict(prefix_len=ints([-2 ** 31, 40])),
                 dict(group_start=ints([-7, 2, 99])), dict(group_start=ints([2, 1, 0])),
                 dict(group_start=ints([5, 6, 7])), dict(q_start=ints([-5, 1, 99, 2])), dict(q_start=ints([4, 3, 2, 1])),
                 dict(seq_len=ints([2 ** 31 - 1, -4, 49])), dict(prefix_table=s.prefix_table[:, :0])):
        s.call(nv, **args, **more)
    nv.device_status(clear=True)
    out, _ = s.call(nv, **args)
    assert torch.equal(out, want) and nv.device_status() == 0


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_nonfinite_query_stays_in_its_row(nv, kernel, dtype, bad):
    s = Shared(nv, [(140, [(5, 1), (60, 40)])], 8, 2, 64, 16, dtype)
    q = s.q.clone()
    q[20, 3, 7] = bad
    out, lse = s.call(nv, q, kernel=getattr(nv, kernel))
    keep = torch.ones((41, 8), dtype=torch.bool, device="cuda")
    keep[20, 3] = False
    assert not torch.isfinite(out[20, 3]).any()
    check_attention(out[keep][None], lse[keep][None], [x[keep][None] for x in s.ref()], dtype)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_zero_tensor_scales(nv, kernel, dtype):
    s = Shared(nv, [(140, [(5, 1), (60, 4)])], 8, 2, 64, 16, dtype)
    s.cache.k_g.zero_()
    out, lse = s.call(nv, kernel=getattr(nv, kernel))
    check_attention(out, lse, s.ref(), dtype)
    s.cache.v_g.zero_()
    assert not s.call(nv, kernel=getattr(nv, kernel))[0].any()


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_streams_and_graphs(nv, kernel, dtype):
    """On a side stream and in graphs: two calls in one, lengths and groups changed between replays."""
    s = Shared(nv, [(100, [(5, 1), (60, 1)]), (300, [(9, 1), (17, 1)])], 8, 2, 64, 16, dtype)
    buf = dict(prefix_len=ints(s.prefix), group_start=ints(s.start), seq_len=ints(s.seqs),
               q_start=ints(starts(s.counts)), kernel=getattr(nv, kernel))
    want, want_lse = s.call(nv, **buf)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = s.call(nv, pdl=False, **buf)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one, one_lse = s.call(nv, pdl=True, **buf)
        two, two_lse = s.call(nv, pdl=True, **buf)
    for change in (0, 1, 0):
        if change:  # the second request of each group alone behind the prefix that is left to it
            buf["seq_len"].copy_(ints([100 + 3, 100 + 60, 300 + 9, 300 + 2]))
        else:
            buf["seq_len"].copy_(ints(s.seqs))
        for x in (one, one_lse, two, two_lse):
            x.fill_(math.nan)
        graph.replay()
        eager, eager_lse = s.call(nv, **buf)
        for o, l in ((one, one_lse), (two, two_lse)):
            assert torch.equal(o, eager) and torch.equal(l, eager_lse)
    assert torch.equal(eager, want) and torch.equal(eager_lse, want_lse)


def test_offsets_past_32_bits(nv):
    """A pool of over 8 GB whose last pages hold a prefix and a request."""
    page, heads, dim = 256, 8, 128
    pages = (9 << 30) // nv.kv_page_bytes(page, heads, dim)
    g = ints([5 / 2688], FP32)
    pool = nv.kv_pool(pages, heads, dim, page)
    pool[-4:] = 0
    cache = nv.KVCache(pool, g, g, page_size=page, head_dim=dim)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((700, heads, dim), generator=gen, device="cuda")
    nv.kv_append(cache, k, k, torch.arange(700, device="cuda") + (pages - 3) * page)
    prefix_table, table = ints([[pages - 3, pages - 2]]), ints([[-1, -1, pages - 1]])
    for rows, kernel in ((1, nv.KERNEL_KV_ROWS), (90, nv.KERNEL_KV_TILE)):
        q = torch.randn((rows, 32, dim), generator=gen, device="cuda").to(BF16)
        out, lse = nv.kv_attention_shared(cache, q, prefix_table, ints([512]), table, ints([700]), return_lse=True,
                                          kernel=kernel)
        keys = shared_keys(cache, prefix_table, [512], [0, 1], table, [700], [rows])
        check_attention(out, lse, attend(q, keys, [rows]), BF16)
        out, lse = nv.kv_cross_attention(cache, q, ints([[pages - 3, pages - 2, pages - 1]]), ints([700]),
                                         return_lse=True, kernel=kernel)
        check_attention(out, lse, attend(q, keys, [rows], causal=False), BF16)


# ---- cross attention -----------------------------------------------------------------------

def run_cross(nv, seqs, counts, hq=8, hkv=2, dim=64, page=16, q_dtype=BF16, scale=None, kernel="KERNEL_AUTO",
              out_dtype=None, seed=0, layers=1, uniform=False, **more):
    cache, table, gen = make(nv, [(0, n) for n in seqs], hkv, dim, page, seed, layers)
    table = table.cuda()
    q = torch.randn((sum(counts), hq + 2 * hkv, dim), generator=gen, device="cuda").to(q_dtype)[:, :hq]
    nv.device_status(clear=True)
    args = dict(dict(max_q=max(counts, default=0)), **more)
    out, lse = nv.kv_cross_attention(cache, q, table, ints(seqs), None if uniform else ints(starts(counts)),
                                     scale=scale, kernel=getattr(nv, kernel), out_dtype=out_dtype, return_lse=True,
                                     **args)
    assert nv.device_status() == 0
    assert out.dtype == (out_dtype or q_dtype)
    ref = attend(q, [table_values(cache, table[r], 0, n) for r, n in enumerate(seqs)], counts, scale, causal=False)
    check_attention(out, lse, ref, q_dtype)
    return cache, table, q, out, lse


LENGTHS = [1, 0, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 1000]


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 64), (64, 256), (128, 128)])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_cross_lengths(nv, kernel, dtype, dim, page, rows):
    """Every boundary, an encoder without states, more rows than states and fewer."""
    run_cross(nv, LENGTHS, [rows] * len(LENGTHS), 8, 2, dim, page, dtype, kernel=kernel)
    run_cross(nv, LENGTHS, [rows] * len(LENGTHS), 2, 2, dim, page, dtype, kernel=kernel, uniform=True, layers=2)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (16, 16), (34, 2), (64, 1), (20, 20)])
def test_cross_head_groups(nv, kernel, dtype, hq, hkv):
    run_cross(nv, [77, 300, 5], [1, 4, 2], hq, hkv, 64, 32, dtype, kernel=kernel, seed=hq)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("counts", [[2, 1, 0, 5], [16, 9], [64, 65, 1], [130, 0, 33], [300], [700, 3, 1, 90]])
@pytest.mark.parametrize("seed", [0, 1])
def test_cross_several_rows(nv, kernel, dtype, counts, seed):
    rng = np.random.default_rng(seed)
    seqs = rng.integers(0, 700, len(counts)).tolist()
    run_cross(nv, seqs, counts, 8, 2, 128, 16, dtype, kernel=kernel, seed=seed)
    run_cross(nv, seqs, counts, 6, 6, 64, 64, dtype, kernel=kernel, seed=seed)


def test_cross_types_scales_hints(nv):
    for q_dtype, out_dtype in ((BF16, FP32), (FP32, BF16)):
        run_cross(nv, [50, 300], [3, 20], 8, 2, 128, 16, q_dtype, out_dtype=out_dtype)
    for scale in (0.3, -0.1, 0.0):
        run_cross(nv, [50, 300], [3, 20], scale=scale)
        run_cross(nv, [50, 300], [3, 20], scale=scale, kernel="KERNEL_KV_TILE")
    for max_q in (0, 1, 1000, None):
        run_cross(nv, [50, 300], [3, 20], max_q=max_q)


def test_cross_long_and_many(nv):
    run_cross(nv, [20011, 0, 3, 4096], [1] * 4, 8, 2, 128, 64)
    run_cross(nv, [9001, 10, 700], [5, 2, 1], 16, 2, 64, 16, FP32)
    run_cross(nv, [9001, 10, 700], [500, 2, 100], 16, 2, 64, 16)
    rng = np.random.default_rng(5)
    run_cross(nv, rng.integers(0, 60, 700).tolist(), [1] * 700, 4, 2, 64, 16)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_cross_is_what_a_last_row_sees(nv, kernel, dtype):
    """A row at a request's last position sees all keys in causal attention, too: both calls hold the
    same reference's bounds (the bits may differ: the keys are shared among the SMs in other pieces)."""
    cache, table, q, out, lse = run_cross(nv, [3000, 15, 200], [1, 1, 1], 8, 2, 64, 16, dtype, kernel=kernel)
    o2, l2 = nv.kv_attention(cache, q, table, ints([3000, 15, 200]), max_q=1, return_lse=True,
                             kernel=getattr(nv, kernel))
    keys = [table_values(cache, table[r], 0, n) for r, n in enumerate((3000, 15, 200))]
    for causal in (False, True):
        ref = attend(q, keys, [1, 1, 1], causal=causal)
        check_attention(out, lse, ref, dtype)
        check_attention(o2, l2, ref, dtype)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_cross_outputs_repeats_and_bad_entries(nv, kernel, dtype):
    seqs, counts = [3000, 0, 70], [3, 1, 40]
    cache, table, q, out, lse = run_cross(nv, seqs, counts, 8, 2, 64, 16, dtype, kernel=kernel)
    args = dict(max_q=40, return_lse=True, kernel=getattr(nv, kernel))
    lens, start = ints(seqs), ints([2, 5, 6, 46])
    q2 = torch.full((50, 8, 64), math.nan, dtype=dtype, device="cuda")
    q2[2:46] = q
    for _ in range(3):
        old = [torch.full((50, 8, 64), math.nan, dtype=dtype, device="cuda") for _ in range(4)]
        del old
        o2, l2 = nv.kv_cross_attention(cache, q2, table, lens, start, **args)
        assert torch.equal(o2[2:46], out) and torch.equal(l2[2:46], lse)
        for rows in (slice(0, 2), slice(46, None)):
            assert not o2[rows].any() and (l2[rows] == -math.inf).all()
    room = torch.full((50, 10, 64), 7.0, dtype=dtype, device="cuda")
    o2, l2 = nv.kv_cross_attention(cache, q2, table, lens, start, out=room[:, 1:9], **args)
    assert torch.equal(o2[2:46], out)
    room[2:46, 1:9] = 7.0
    assert (room == 7.0).all()
    broken = table.clone()
    broken[0, 3] = -1
    nv.device_status(clear=True)
    o2, l2 = nv.kv_cross_attention(cache, q2, broken, lens, start, **args)
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE and torch.equal(o2[6:46], out[4:])
    nv.kv_cross_attention(cache, q2, table[:, :3], lens, start, **args)
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, l3 = nv.kv_cross_attention(cache, q2, table, lens, start, pdl=True, **args)
    o3.fill_(math.nan)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o3[2:46], out) and torch.equal(l3[2:46], lse)


# ---- refusals of the binding ------------------------------------------------------------------

def test_binding_refusals(nv):
    s = Shared(nv, [(100, [(5, 1), (60, 1)]), (30, [(9, 1)])], 8, 2, 64, 16, FP32)
    ok = dict(cache=s.cache, q=s.q, prefix_table=s.prefix_table, prefix_len=ints(s.prefix), block_table=s.table,
              seq_len=ints(s.seqs), group_start=ints(s.start))
    for change in (dict(prefix_table=s.prefix_table[:1]), dict(prefix_table=s.prefix_table.long()),
                   dict(prefix_table=s.prefix_table.cpu()), dict(prefix_table=None), dict(prefix_len=None),
                   dict(prefix_len=ints(s.prefix, torch.int64)), dict(prefix_len=ints([1])), dict(group_start=None),
                   dict(group_start=ints([0, 3])), dict(group_start=ints(s.start).cpu()),
                   dict(group_start=ints(s.start, torch.int64)), dict(q=s.q.half()), dict(q=s.q[:2]),
                   dict(block_table=s.table[:1]), dict(seq_len=ints(s.seqs, torch.int64)), dict(out=s.q[:1]),
                   dict(out_dtype=torch.float16), dict(workspace=torch.zeros(100, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            nv.kv_attention_shared(**{**ok, **change})
    for change in (dict(kernel=77), dict(kernel=nv.KERNEL_KV_TILE), dict(scale=math.nan)):
        with pytest.raises(nv.Nvfp4Error):
            nv.kv_attention_shared(**{**ok, **change})
    with pytest.raises(TypeError):
        nv.kv_attention_shared(**ok, window=4)
    cross = dict(cache=s.cache, q=s.q, block_table=s.table, seq_len=ints([1, 1, 1]))
    for change in (dict(q=s.q.cpu()), dict(q=s.q[:, :7]), dict(block_table=s.table.T), dict(seq_len=ints([1.0], FP32)),
                   dict(q_start=ints([0, 1])), dict(q=s.q[:2]), dict(out=s.q.half()), dict(out_dtype=torch.float64)):
        with pytest.raises(ValueError):
            nv.kv_cross_attention(**{**cross, **change})
    for change in (dict(kernel=77), dict(kernel=nv.KERNEL_KV_TILE), dict(scale=math.nan), dict(max_q=-1)):
        with pytest.raises(nv.Nvfp4Error):
            nv.kv_cross_attention(**{**cross, **change})
    with pytest.raises(TypeError):
        nv.kv_cross_attention(**cross, window=4)


# ---- a step of all of them together ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_decode_step(nv, dtype):
    """Two prompts sampled several times: tables, the rotating append and attention behind the
    prefixes, three steps; then cross attention to states appended without a rotation."""
    page, hq, hkv, dim, rot = 16, 8, 2, 64, 64
    prefix, members = [37, 70], [3, 2]
    reqs = sum(members)
    gen = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(dtype)  # noqa: E731
    a = torch.arange(200, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    rotary = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    cache = nv.KVCache(nv.kv_pool(60, hkv, dim, page), ints([6 / 2688], FP32), ints([5 / 2688], FP32), page_size=page,
                       head_dim=dim)
    cache.pool.fill_(255)
    free = torch.randperm(60, generator=gen, device="cuda").to(torch.int32)
    # the prompts, once each
    prefix_table = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
    t = nv.kv_tables(ints([0, 0]), ints(prefix), free, ints([0]), prefix_table, page_size=page, tokens=sum(prefix))
    rows = rand(sum(prefix), hq + 2 * hkv, dim)
    q = nv.kv_append_rotary(cache, rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], t.slots, t.positions, rotary)
    prompts = nv.kv_attention(cache, q, prefix_table, t.seq_len, t.q_start, max_q=70)
    check_attention(prompts, None, attend(q, [table_values(cache, prefix_table[g], 0, n) for g, n in enumerate(prefix)],
                                          prefix), dtype)
    # every request goes on in its own page behind its prompt: a partial last page is its own from here on
    lens = ints([p // page * page for p, m in zip(prefix, members) for _ in range(m)])
    shared = [p // page * page for p in prefix]  # what is shared ends with a page; the rest is appended again
    table = torch.full((reqs, 8), -1, dtype=torch.int32, device="cuda")
    group_start, head = ints([0, 3, 5]), t.free_head
    for step, count in enumerate(([5, 5, 5, 6, 6], [1] * 5, [3, 1, 2, 1, 1])):
        t = nv.kv_tables(lens, ints(count), free, head, table, page_size=page, tokens=sum(count) + 2)
        rows = rand(sum(count) + 2, hq + 2 * hkv, dim)
        k = rows[:, hq:hq + hkv]
        q = nv.kv_append_rotary(cache, rows[:, :hq], k, rows[:, hq + hkv:], t.slots, t.positions, rotary)
        assert torch.equal(q.cpu(), rotated(rows[:, :hq], t.positions, rotary, False).to(dtype))
        out, lse = nv.kv_attention_shared(cache, q, prefix_table, ints(shared), table, t.seq_len, t.q_start,
                                          group_start=group_start, max_q=max(count), return_lse=True)
        seqs = t.seq_len.tolist()
        keys = shared_keys(cache, prefix_table, shared, [0, 3, 5], table, seqs, count)
        used = sum(count)
        check_attention(out[:used], lse[:used], attend(q[:used], keys, count), dtype)
        assert not out[used:].any()
        lens, head = t.seq_len.clone(), t.free_head.clone()
    # an encoder's states for the same requests, in pages of the same pool
    src = [20, 1, 0, 33, 16]
    states = torch.full((reqs, 3), -1, dtype=torch.int32, device="cuda")
    s = nv.kv_tables(ints([0] * reqs), ints(src), free, head, states, page_size=page, tokens=sum(src))
    kv = rand(sum(src), 2 * hkv, dim)
    nv.kv_append(cache, kv[:, :hkv], kv[:, hkv:], s.slots)
    out, lse = nv.kv_cross_attention(cache, q[:used], states, s.seq_len, t.q_start, max_q=3, return_lse=True)
    check_attention(out, lse, attend(q[:used], [table_values(cache, states[r], 0, n) for r, n in enumerate(src)],
                                     [3, 1, 2, 1, 1], causal=False), dtype)
    assert nv.device_status() == 0
    kk, _ = page_values(cache.pool[states[0, 0].long()][None], page, dim)
    assert (kk[0].transpose(0, 1) * cache.k_g.double() - kv[:page, :hkv].double()).abs().max() < 1.0


# ---- references that rise --------------------------------------------------------------------

def rising(nv, cache, table, lo, hi, gen, step=1 / 100, down=False):
    """Keys whose scores grow along the tokens [lo, hi) of a table's row; returns the direction."""
    page, heads, dim = cache.page_size, cache.num_kv_heads, cache.head_dim
    base = torch.randn((dim,), generator=gen, device="cuda")
    i = torch.arange(hi - lo, device="cuda")
    k = ((hi - lo - 1 - i if down else i)[:, None, None] * (base * step)).expand(-1, heads, -1).contiguous()
    v = torch.randn((hi - lo, heads, dim), generator=gen, device="cuda")
    at = lo + i
    slots = table[at // page].long() * page + at % page
    nv.kv_append(cache, k, v, slots)
    return base, k


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("dim", [64, 128])
def test_cross_growing_scores(nv, kernel, dtype, dim):
    """Scores of hundreds that rise (or fall) along the states, whole requests and cut ones: what was summed
    is rescaled again and again, also inside a block and where only a few of a warp's rows rise."""
    n = 1900
    for down in (False, True):
        cache, table, gen = make(nv, [(0, n)], 1, dim, 16)
        table = table.cuda()
        base, k = rising(nv, cache, table[0], 0, n, gen, 1 / 300, down)
        cache.k_g.copy_(nv.global_scale(k))
        nv.kv_append(cache, k, torch.randn((n, 1, dim), generator=gen, device="cuda"),
                     table[0, torch.arange(n, device="cuda") // 16].long() * 16 + torch.arange(n, device="cuda") % 16)
        q = torch.randn((70, 4, dim), generator=gen, device="cuda")
        q[::3] += base * 10
        q[1::7] -= base * 5
        q = q.to(dtype)
        for ws in (None, False):
            out, lse = nv.kv_cross_attention(cache, q, table, ints([n]), return_lse=True, kernel=getattr(nv, kernel),
                                             workspace=ws)
            ref = attend(q, [table_values(cache, table[0], 0, n)], [70], causal=False)
            check_attention(out, lse, ref, dtype)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_shared_growing_scores(nv, kernel, dtype):
    """The same through a prefix into the own keys of prompts behind it."""
    s = Shared(nv, [(1000, [(300, 200), (90, 3)])], 4, 1, 64, 16, dtype)
    s.cache.k_g.fill_(5.0 / 300 * 1000 / 2688)
    base, _ = rising(nv, s.cache, s.prefix_table[0], 0, 1000, s.gen, 1 / 300)
    for r in range(2):
        rising(nv, s.cache, s.table[r], 1000, s.seqs[r], s.gen, 1 / 100, down=bool(r))
    q = s.q.float()
    q[::3] += base * 8
    q = q.to(dtype)
    out, lse = s.call(nv, q, kernel=getattr(nv, kernel))
    check_attention(out, lse, s.ref(q=q), dtype)


@pytest.mark.parametrize("name", ["KERNEL_KV_ROWS", "KERNEL_KV_TILE"])
def test_cross_probabilities_are_rounded_once(nv, name):
    """One f16 rounding of each probability (the bound's 2^-11), also where the reference rises inside a
    block: 128 keys of score 0, 64 about 2^7 times as probable with values of +1, then 16 about 2^9
    times with values of -1, so that the rest of the two sums is what roundings leave."""
    n, rows, group = 320, 64, 64
    unit = 1.4426950408889634  # scores below are in powers of two
    cache, table, gen = make(nv, [(0, n)], 1, 64, 16)
    table = table.cuda()
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
    q = torch.zeros((rows, group, 64), device="cuda")
    rand = lambda: torch.rand((rows, group), generator=gen, device="cuda")  # noqa: E731
    q[..., 1], q[..., 17] = rand(), rand()
    q[..., 0] = (7.0 + 0.08 * rand() - 0.5 * q[..., 1]) / 6.0
    q[..., 16] = (8.93 + 0.069 * rand() - 0.5 * q[..., 17]) / 6.0
    q[..., 32] = 10.0
    q = q.to(BF16)
    out, lse = nv.kv_cross_attention(cache, q, table, ints([n]), scale=1.0 / unit, return_lse=True,
                                     kernel=getattr(nv, name), workspace=False)
    ref = attend(q, [table_values(cache, table[0], 0, n)], [rows], 1.0 / unit, causal=False)
    check_attention(out, lse, ref, BF16)


@pytest.mark.parametrize("name", ["KERNEL_KV_ROWS", "KERNEL_KV_TILE"])
@pytest.mark.parametrize("form", ["causal", "cross", "prefix", "behind"])
def test_small_probabilities_stay_where_the_reference_rises(nv, form, name):
    """A probability is held to 2^-32 of its row's largest (the bound's reach) also where the reference rises
    far inside a block: 64 keys with values of 1, then 16 keys that are 2^18 to 2^36 times as probable, with
    values of 0, so that the output is what is left of the first ones."""
    n, rows, group = 384, 64, 64
    unit = 1.4426950408889634  # scores below are in powers of two
    cache, table, gen = make(nv, [(0, n)], 1, 64, 16)
    table = table.cuda()
    k = torch.zeros((n, 1, 64), device="cuda")
    k[128:192, 0, 0] = 6.0
    k[192:208, 0, 16] = 6.0
    k[208:, 0, 32] = -6.0  # as good as unseen
    v = torch.zeros((n, 1, 64), device="cuda")
    v[128:192] = 1.0
    cache.k_g.fill_(1.0)
    cache.v_g.fill_(1.0)
    slots = table[0, :n // 16].long().repeat_interleave(16) * 16 + torch.arange(n, device="cuda") % 16
    nv.kv_append(cache, k, v, slots)
    q = torch.zeros((rows, group, 64), device="cuda")
    q[..., 0] = 30.0 / 6.0
    q[..., 16] = (48.0 + 18.0 * torch.rand((rows, group), generator=gen, device="cuda")) / 6.0
    q[..., 32] = 10.0
    q = q.to(BF16)
    # (no workspace: a request's keys stay with one SM, in order)
    args = dict(scale=1.0 / unit, return_lse=True, kernel=getattr(nv, name), workspace=False)
    if form == "causal":
        out, lse = nv.kv_attention(cache, q, table, ints([n]), **args)
    elif form == "cross":
        out, lse = nv.kv_cross_attention(cache, q, table, ints([n]), **args)
    else:
        out, lse = nv.kv_attention_shared(cache, q, table, ints([320 if form == "prefix" else 16]), table, ints([n]),
                                          **args)
    ref = attend(q, [table_values(cache, table[0], 0, n)], [rows], 1.0 / unit, causal=form != "cross")
    check_attention(out, lse, ref, BF16)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_pages_and_layers(nv, kernel, dtype):
    """Strided pages (one pool for several layers), every page size, prefixes that end inside a page."""
    for page in (16, 32, 64, 128, 256):
        run_shared(nv, [(page + 5, [(page * 2, 1), (3, 3)]), (page, [(1, 1)])], 8, 4, 128, page, dtype, kernel=kernel,
                   layers=3)


def test_starts_that_go_back_lead_nowhere(nv):
    """A request's rows reach over those of its group: what the first pass has not written is not followed
    (results mean nothing there); the next call is right."""
    s = Shared(nv, [(300, [(5, 1), (20, 3)]), (40, [(9, 2)])], 8, 2, 64, 16, BF16)
    want, _ = s.call(nv)
    for fill in (math.nan, 1e30, 2.0, 0.0):
        old = [torch.full((1 << 22,), fill, device="cuda") for _ in range(8)]  # memory that the call may take
        old += [torch.full((1 << 22,), 2 ** 31 - 1, dtype=torch.int32, device="cuda") for _ in range(4)]
        del old
        for start in ([0, 5, 2, 6], [0, 6, 1, 4], [2, 6, 0, 6], [0, 1, 0, 6]):
            for kernel in (nv.KERNEL_KV_ROWS, nv.KERNEL_KV_TILE):
                s.call(nv, q_start=ints(start), kernel=kernel)
    torch.cuda.synchronize()
    nv.device_status(clear=True)
    out, _ = s.call(nv)
    assert torch.equal(out, want) and nv.device_status() == 0


# ---- calls beside one another -----------------------------------------------------------------

@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_two_streams_and_two_graphs(nv, kernel, dtype):
    """Calls of one cache on two streams at once, and two graphs replayed beside them, with the default
    workspaces and scratch: the bits of calls that run alone."""
    s = Shared(nv, [(3000, [(50 + i, 1) for i in range(6)] + [(70, 40)]), (500, [(9, 2)])], 8, 2, 64, 16, dtype)
    args = dict(kernel=getattr(nv, kernel))
    table, lens, start = s.args["prefix_table"], ints([3000, 500]), ints([0, 46, 48])

    def both():
        a, al = s.call(nv, **args)
        b, bl = nv.kv_cross_attention(s.cache, s.q, table, lens, start, max_q=46, return_lse=True, **args)
        return a, al, b, bl

    want = [x.clone() for x in both()]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, results = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(both())
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for x in itertools.chain(*results):
            x.fill_(math.nan)
        torch.cuda.synchronize()
        for i in range(4):
            with torch.cuda.stream(streams[i % 2]):
                got.append(both())
                if i < 2:
                    graphs[i].replay()
        torch.cuda.synchronize()
        for r in got + results:
            for x, w in zip(r, want):
                assert torch.equal(x, w)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
def test_tables_with_strides(nv, kernel, dtype):
    """Tables that are parts of wider ones, with more columns than are used."""
    s = Shared(nv, [(100, [(5, 1), (60, 9)]), (33, [(9, 2)])], 8, 2, 64, 16, dtype)
    args = dict(kernel=getattr(nv, kernel))
    want, want_lse = s.call(nv, **args)
    wide = []
    for t in (s.prefix_table, s.table):
        w = torch.full((t.shape[0], t.shape[1] + 13), -5, dtype=torch.int32, device="cuda")
        w[:, 4:4 + t.shape[1]] = t
        wide.append(w[:, 4:4 + t.shape[1]])
    out, lse = s.call(nv, prefix_table=wide[0], block_table=wide[1], **args)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    one, one_lse = nv.kv_cross_attention(s.cache, s.q[:2], wide[0], ints(s.prefix), max_q=1, return_lse=True, **args)
    two, two_lse = nv.kv_cross_attention(s.cache, s.q[:2], s.prefix_table, ints(s.prefix), max_q=1, return_lse=True,
                                         **args)
    assert torch.equal(one, two) and torch.equal(one_lse, two_lse)


def test_more_groups_than_a_warp_takes(nv):
    """More than 32 groups with long prefixes: shares of one list, cut anywhere."""
    for kernel, dtype in KERNELS:
        run_shared(nv, [(700 + 13 * g, [(5 + g, 1), (9, 2)]) for g in range(40)], 8, 2, 64, 16, dtype, kernel=kernel)
        run_shared(nv, [(9000, [(5, 1)])] + [(g, [(5 + g, 3)]) for g in range(1, 33)], 8, 2, 64, 64, dtype, kernel=kernel)


@pytest.mark.parametrize("kernel,dtype", KERNELS)
@pytest.mark.parametrize("rows", [1, 40])
def test_in_place(nv, kernel, dtype, rows):
    """The output over the queries (heads of a wider row), with and without cut items: the same bits."""
    s = Shared(nv, [(9000, [(50, rows), (700, rows)]), (300, [((200,), rows), (1 + rows, rows)])], 8, 2, 128, 16, dtype)
    args = dict(kernel=getattr(nv, kernel))
    table, lens, start = s.args["prefix_table"], ints([9000, 300]), ints([0, 2 * rows, 4 * rows])
    for call in (lambda q, **more: s.call(nv, q, **args, **more),
                 lambda q, **more: nv.kv_cross_attention(s.cache, q, table, lens, start, return_lse=True, **args, **more)):
        want, want_lse = call(s.q)
        wide = torch.cat((s.q, s.q, s.q), 1)
        q, rest = wide[:, 8:16], wide[:, 16:].clone()
        out, lse = call(q, out=q)
        assert out.data_ptr() == q.data_ptr()
        assert torch.equal(q, want) and torch.equal(lse, want_lse)
        assert torch.equal(wide[:, :8], s.q) and torch.equal(wide[:, 16:], rest)
        with pytest.raises(nv.Nvfp4Error):
            call(q, out=wide[:, 9:17])


@pytest.mark.parametrize("kernel", ["KERNEL_AUTO", "KERNEL_KV_TILE"])
@pytest.mark.parametrize("rows,reqs", [(7, 40), (40, 60)])
def test_in_place_beside_rows_inside_the_prefix(nv, kernel, rows, reqs):
    """Requests with rows inside their prefix between such that share it, the output over the queries: the
    prefix's pass takes rows of both side by side, and the first ones' outputs must not come under it.
    Their queries are large, so that a row read half old and half new would move its neighbours'
    references and with them their last bits.  (40 rows of 60 requests: the own keys on the tcgen05 kernel by
    the library's choice too.)"""
    group = [((50 + 9 * r,), rows) if r % 2 else (rows + 3 * r, rows) for r in range(reqs)]
    s = Shared(nv, [(9000, group), (5000, group[::-1])], 8, 2, 128, 16, BF16)
    q = s.q.clone().view(-1, rows, 8, 128)
    q[1:reqs:2] *= 40.0
    q[reqs::2] *= 40.0  # the second group begins with one of them (reqs is even)
    q = q.flatten(0, 1)
    args = dict(kernel=getattr(nv, kernel))
    want, want_lse = s.call(nv, q, **args)
    assert not torch.equal(want, q)
    check_attention(want, want_lse, s.ref(q=q), BF16)
    for _ in range(30):
        mine = q.clone()
        out, lse = s.call(nv, mine, out=mine, **args)
        assert out.data_ptr() == mine.data_ptr()
        assert torch.equal(mine, want) and torch.equal(lse, want_lse)
