"""The rotating append on the GPU: queries and appended bytes against the rotation's rounding
steps on the CPU and the oracle's quantiser, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from kv_rows_helpers import rotated

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


def angles(rows, rot, base=10000.0):
    a = torch.arange(rows, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def make_cache(nv, pages, heads, dim, page, kg, vg, layers=1, layer=0):
    whole = nv.kv_pool(pages * layers, heads, dim, page)
    whole.random_(0, 256)
    pool = whole.view(pages, layers, heads, -1)[:, layer]
    return nv.KVCache(pool, kg, vg, page_size=page, head_dim=dim), whole


def written(cache, whole, layers, layer, k, v, slots):
    """The pool after the append of k, v [tokens, heads, dim] float32 (CPU) by the oracle's recipe."""
    page, dim, heads = cache.page_size, cache.head_dim, cache.num_kv_heads
    want = whole.cpu().clone()
    mine = want.view(-1, layers, heads, whole.shape[-1])[:, layer]
    half, block = page * dim // 2, page * dim // 16
    for part, (x, g) in enumerate(((k, cache.k_g), (v, cache.v_g))):
        tokens = x.shape[0]
        q, s = oracle.quantize(x.contiguous().numpy().reshape(tokens * heads, dim), np.float32(g.item()))
        q, s = torch.from_numpy(q).view(tokens, heads, -1), torch.from_numpy(s).view(tokens, heads, -1)
        for t, slot in enumerate(slots.tolist()):
            if slot < 0:
                continue
            p, o = divmod(slot, page)
            mine[p, :, part * half + o * dim // 2:part * half + (o + 1) * dim // 2] = q[t]
            at = 2 * half + part * block + o * dim // 16
            mine[p, :, at:at + dim // 16] = s[t]
    return want


def check(nv, dtype, hq, heads, dim, page, tokens, rot, interleaved, layers=1, rows_of=None, seed=0, span=300,
          magnitudes=True, out=None, pdl=False):
    gen = torch.Generator(device="cuda").manual_seed(seed + dim + rot)
    rows = torch.randn((tokens, hq + 2 * heads + 1, dim), generator=gen, device="cuda")
    if magnitudes:
        rows *= torch.exp2(torch.randint(-14, 4, (tokens, hq + 2 * heads + 1, 1), generator=gen, device="cuda"))
        rows[::5, :, :16] = 0.0
        rows[1::5, :, :16] = -0.0
    rows = rows.to(dtype)
    if rows_of is not None:
        rows = rows_of(rows)
    q, k, v = rows[:, :hq], rows[:, hq:hq + heads], rows[:, hq + heads:hq + 2 * heads]
    rotary = angles(span, rot)
    pos = torch.randint(0, span, (tokens,), generator=gen, device="cuda").to(torch.int32)
    pages = -(-tokens // page) + 5
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:tokens].contiguous()
    slots[3::7] = -1
    cache, whole = make_cache(nv, pages, heads, dim, page, ints([0.0011], FP32), ints([0.0002], FP32), layers, layers - 1)
    want_q = rotated(q, pos, rotary, interleaved).to(dtype)
    want = written(cache, whole, layers, layers - 1, rotated(k, pos, rotary, interleaved), v.float().cpu(), slots)
    nv.device_status(clear=True)
    got = nv.kv_append_rotary(cache, q, k, v, slots, pos, rotary, interleaved=interleaved,
                              out=out(q) if out else None, pdl=pdl)
    assert nv.device_status() == 0
    assert got.dtype == dtype and got.shape == q.shape
    assert torch.equal(got.cpu().view(torch.int16 if dtype == BF16 else torch.int32),
                       want_q.view(torch.int16 if dtype == BF16 else torch.int32))
    assert torch.equal(whole.cpu(), want)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 96), (128, 64), (128, 32), (64, 64), (64, 32)])
def test_rotations(nv, dtype, interleaved, dim, rot):
    check(nv, dtype, 8, 2, dim, 16, 37, rot, interleaved)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("hq,heads,dim,page,tokens,layers",
                         [(32, 8, 128, 16, 1, 1), (32, 8, 128, 64, 8, 2), (7, 1, 64, 16, 3, 1), (3, 3, 64, 32, 65, 1),
                          (5, 2, 128, 128, 33, 3), (1, 1, 64, 256, 2, 1), (64, 32, 128, 256, 40, 1)])
def test_shapes(nv, dtype, hq, heads, dim, page, tokens, layers):
    """One token to a few, strided pages, query heads that are no multiple of the kv heads."""
    check(nv, dtype, hq, heads, dim, page, tokens, dim, False, layers)
    check(nv, dtype, hq, heads, dim, page, tokens, 32, True, layers)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("hq,heads,tokens", [(13, 2, 4001), (32, 8, 1500), (1, 1, 20011)])
def test_many_tokens(nv, dtype, hq, heads, tokens):
    """Enough for several query heads a thread, also where their number is no multiple of that."""
    check(nv, dtype, hq, heads, 64, 64, tokens, 64, False)
    check(nv, dtype, hq, heads, 64, 64, tokens, 32, True)


@pytest.mark.parametrize("shift,extra", [(4, 0), (0, 4), (4, 4)])
@pytest.mark.parametrize("tokens", [5, 3000])
def test_rows_on_8_byte_boundaries(nv, shift, extra, tokens):
    def moved(rows):
        n, h, d = rows.shape
        flat = torch.zeros(n * (h * d + extra) + 8, dtype=rows.dtype, device="cuda")
        view = flat[shift:].as_strided((n, h, d), (h * d + extra, d, 1))
        view.copy_(rows)
        return view
    check(nv, BF16, 8, 2, 128, 16, tokens, 128, False, rows_of=moved)
    check(nv, BF16, 8, 2, 64, 16, tokens, 32, True, rows_of=moved)


def test_outputs_in_place_and_in_slices(nv):
    check(nv, BF16, 8, 2, 128, 16, 300, 128, False, out=lambda q: q)
    check(nv, FP32, 8, 2, 64, 16, 3, 32, True, out=lambda q: q)
    check(nv, FP32, 8, 2, 64, 16, 30, 64, False, out=lambda q: torch.empty((30, 11, 64), device="cuda")[:, 2:10])
    room = torch.full((30, 11, 64), 7.0, device="cuda")
    check(nv, FP32, 8, 2, 64, 16, 30, 64, False, out=lambda q: room[:, 2:10])
    assert (room[:, :2] == 7).all() and (room[:, 10:] == 7).all()


def test_without_queries_it_is_the_append_of_turned_keys(nv):
    """And with angles of zero, the plain append."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((50, 2, 64), generator=gen, device="cuda") for _ in "kv")
    g = ints([0.002], FP32)
    slots = torch.randperm(64, generator=gen, device="cuda")[:50].contiguous()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    for rotary in (angles(60, 64), angles(60, 64)[:1].expand(60, 64).contiguous()):
        a, pool_a = make_cache(nv, 4, 2, 64, 16, g, g)
        b, pool_b = make_cache(nv, 4, 2, 64, 16, g, g)
        pool_b.copy_(pool_a)
        assert nv.kv_append_rotary(a, None, k, v, slots, pos, rotary) is None
        nv.kv_append(b, rotated(k, pos, rotary, False).cuda(), v, slots)
        assert torch.equal(pool_a, pool_b)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_bad_positions_and_slots(nv, dtype):
    """Positions outside the table: zeros, nothing appended, reported; padding is not reported."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((6, 4, 64), generator=gen, device="cuda").to(dtype)
    k, v = q[:, :2], q[:, 2:]
    g = ints([0.002], FP32)
    cache, whole = make_cache(nv, 4, 2, 64, 16, g, g)
    rotary = angles(10, 64)
    before = whole.clone()
    for slots, pos, status, zero in (
            ([-1, -1, -1, -1, -1, -1], [0, 10, -1, 5, 2 ** 31 - 1, -2 ** 31], 0, [1, 2, 4, 5]),
            ([3, -1, -1, -1, -1, -1], [10, 0, 0, 0, 0, 0], nv.DEVICE_KV_RANGE, [0]),
            ([-1, -1, 5, -1, -1, -1], [1, 1, -1, 1, 1, 1], nv.DEVICE_KV_RANGE, [2]),
            ([64, -2, 1 << 40, -(1 << 40), -1, -1], [1] * 6, nv.DEVICE_KV_RANGE, [])):
        nv.device_status(clear=True)
        got = nv.kv_append_rotary(cache, q, k, v, ints(slots, torch.int64), ints(pos), rotary)
        assert nv.device_status(clear=True) == status
        assert torch.equal(whole, before)
        safe = torch.tensor(pos).clamp(0, 9)
        want = rotated(q, safe, rotary, False).to(dtype)
        want[zero] = 0
        assert torch.equal(got.cpu(), want)
    # no positions at all
    nv.device_status(clear=True)
    got = nv.kv_append_rotary(cache, q, k, v, ints([0, 1, 2, 3, 4, 5], torch.int64), ints([0] * 6), rotary[:0])
    assert nv.device_status(clear=True) == nv.DEVICE_KV_RANGE and not got.any() and torch.equal(whole, before)
    assert nv.kv_append_rotary(cache, q[:0], k[:0], v[:0], ints([], torch.int64), ints([]), rotary).shape == (0, 4, 64)


def test_strided_table_of_angles(nv):
    gen = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn((9, 4, 64), generator=gen, device="cuda")
    g = ints([0.002], FP32)
    cache, whole = make_cache(nv, 4, 2, 64, 16, g, g)
    wide = torch.zeros((30, 100), device="cuda")
    wide[:, 4:68] = angles(30, 64)
    pos, slots = ints(list(range(20, 29))), torch.arange(9, device="cuda")
    got = nv.kv_append_rotary(cache, q, q[:, :2], q[:, 2:], slots, pos, wide[:, 4:68])
    want = nv.kv_append_rotary(cache, q, q[:, :2], q[:, 2:], slots, pos, angles(30, 64))
    assert torch.equal(got, want)
    with pytest.raises(nv.Nvfp4Error):
        nv.kv_append_rotary(cache, q, q[:, :2], q[:, 2:], slots, pos, wide[:, 3:67])  # not on 16 bytes


def test_offsets_past_32_bits(nv):
    """A pool of over 8 GB, rows of queries over 8 GB apart, a table of angles of over 8 GB."""
    page, heads, dim = 256, 8, 128
    pages = (9 << 30) // nv.kv_page_bytes(page, heads, dim)
    g = ints([5 / 2688], FP32)
    whole = nv.kv_pool(pages, heads, dim, page)
    cache = nv.KVCache(whole, g, g, page_size=page, head_dim=dim)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = (9 << 30) // 512
    rotary = torch.zeros((rows, dim), device="cuda")
    rotary[-300:] = angles(300, dim)
    x = torch.randn((3, 24, dim), generator=gen, device="cuda")
    stride = (5 << 30) // 4
    far = torch.empty(2 * stride + 24 * dim, device="cuda").as_strided((3, 24, dim), (stride, dim, 1))
    far.copy_(x)
    q, k, v = far[:, :8], far[:, 8:16], far[:, 16:]
    pos = ints([rows - 1, rows - 300, rows - 77])
    slots = ints([pages * page - 1, (pages - 2) * page, 5], torch.int64)
    got = nv.kv_append_rotary(cache, q, k, v, slots, pos, rotary, out=q)
    assert got.data_ptr() == q.data_ptr()
    small = pos - (rows - 300)
    assert torch.equal(got.cpu(), rotated(x[:, :8], small, angles(300, dim), False))
    turned = rotated(x[:, 8:16], small, angles(300, dim), False)
    for t, slot in enumerate(slots.tolist()):
        p, o = divmod(slot, page)
        codes, scales = oracle.quantize(turned[t].numpy(), np.float32(g.item()))
        assert torch.equal(whole[p, :, o * 64:(o + 1) * 64].cpu(), torch.from_numpy(codes))
        at = page * dim + o * 8
        assert torch.equal(whole[p, :, at:at + 8].cpu(), torch.from_numpy(scales))


@pytest.mark.parametrize("scale", [2.0 ** -130, 2.0 ** 105])
def test_extreme_magnitudes(nv, scale):
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((40, 2, 64), generator=gen, device="cuda") * scale
    pos, slots = torch.arange(40, dtype=torch.int32, device="cuda"), torch.arange(40, device="cuda")
    rotary = angles(40, 64)
    turned = rotated(x, pos, rotary, False)
    g = nv.global_scale(turned.cuda())
    cache, whole = make_cache(nv, 3, 2, 64, 16, g, g)
    want = written(cache, whole, 1, 0, turned, x.cpu(), slots)
    got = nv.kv_append_rotary(cache, x, x, x, slots, pos, rotary)
    assert torch.equal(got.cpu(), turned) and torch.equal(whole.cpu(), want)


def test_streams_and_graphs(nv):
    gen = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn((20, 8, 64), generator=gen, device="cuda").to(BF16)
    g = ints([0.002], FP32)
    cache, whole = make_cache(nv, 4, 2, 64, 16, g, g)
    pos, slots, rotary = ints(list(range(20))), torch.arange(20, device="cuda"), angles(64, 64)

    def step():
        return nv.kv_append_rotary(cache, q, q[:, :2], q[:, 2:4], slots, pos, rotary, pdl=True)

    want, pool = step().clone(), whole.clone()
    whole.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for shift in (0, 7):
        pos.add_(shift)  # the graph reads the positions as they are then
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), rotated(q, pos, rotary, False).to(BF16))
    pos.sub_(7)
    whole.copy_(pool)
    step()
    assert torch.equal(whole, pool)


def test_binding_refusals(nv):
    gen = torch.Generator(device="cuda").manual_seed(8)
    rows = torch.randn((5, 12, 64), generator=gen, device="cuda")
    g = ints([0.002], FP32)
    cache, whole = make_cache(nv, 4, 2, 64, 16, g, g)
    before = whole.clone()
    ok = dict(cache=cache, q=rows[:, :8], k=rows[:, 8:10], v=rows[:, 10:], slots=torch.arange(5, device="cuda"),
              positions=ints([0, 1, 2, 3, 4]), rotary=angles(10, 64))
    for change in (dict(q=ok["q"].half()), dict(q=ok["q"].to(BF16)), dict(q=ok["q"].cpu()), dict(q=ok["q"][:4]),
                   dict(q=ok["q"][:, :, :32]), dict(q=ok["q"].transpose(0, 1)), dict(k=ok["k"][:, :1]),
                   dict(k=None), dict(v=ok["v"].to(BF16)), dict(slots=ok["slots"].int()), dict(slots=ok["slots"][:4]),
                   dict(positions=ok["positions"].long()), dict(positions=ok["positions"][:4]),
                   dict(rotary=ok["rotary"].double()), dict(rotary=ok["rotary"][0]), dict(rotary=ok["rotary"].cpu()),
                   dict(rotary=angles(10, 64).T), dict(rotary=angles(10, 128)), dict(out=ok["q"][:4]),
                   dict(out=ok["q"].to(BF16)), dict(q=None, out=ok["q"]), dict(positions=None)):
        with pytest.raises(ValueError):
            nv.kv_append_rotary(**{**ok, **change})
    for change in (dict(rotary=angles(10, 48)), dict(rotary=angles(10, 16)),
                   # outputs over what is read meanwhile
                   dict(out=rows[:, 1:9]), dict(out=rows[:, 3:11]), dict(out=rows[:, 4:]),
                   dict(k=rows[:, :2]), dict(k=rows[:, 6:8], out=ok["q"])):
        if "k" in change and "out" not in change:
            change = dict(change, out=ok["q"])
        with pytest.raises(nv.Nvfp4Error):
            nv.kv_append_rotary(**{**ok, **change})
    assert torch.equal(whole, before) and nv.device_status() == 0
