"""The entry points of the rotating append, of attention behind shared prefixes and of cross
attention refuse what they cannot take, on the host, before any launch.  CPU only: the
calls below never reach a kernel."""
import struct

import pytest
import torch

import nvfp4_w4a4_decode_gb300 as nv
from nvfp4_w4a4_decode_gb300 import build as nvbuild
from test_kv_abi import BAD_CACHES, FAKE, INVALID, OK, UNSUPPORTED, attention, cache

CUDA = 3
_ROTARY = struct.Struct("@PqqPqPqPqqPPPqqii")  # nvfp4_kv_rotary_args
_PREFIXES = struct.Struct("@PqqPPqPN")         # nvfp4_kv_prefixes
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return nv.library()


def rotary(**change):
    """Operands in memory of their own: 3 tokens of 32 / 8 heads of 128 in FP32."""
    d = dict(q=FAKE, q_stride=4096, q_heads=32, q_out=FAKE + MB, q_out_stride=4096, k=FAKE + 2 * MB, k_stride=1024,
             v=FAKE + 3 * MB, v_stride=1024, tokens=3, slots=FAKE + 4 * MB, positions=FAKE + 5 * MB,
             rotary=FAKE + 6 * MB, rows=100, row_stride=128, rot=128, interleaved=0)
    d.update(change)
    return _ROTARY.pack(*(v or 0 for v in d.values()))


def far_cache(**change):
    """A cache whose memory lies behind the operands above."""
    return cache(**{**dict(pool=FAKE + 16 * MB, k_g=FAKE + 14 * MB, v_g=FAKE + 15 * MB), **change})


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_refusals(lib, change, status):
    c = cache(**change)
    assert lib.nvfp4_kv_append_rotary(c, rotary(), 0, None) == status
    assert lib.nvfp4_kv_cross_attention(c, attention(), 0, None, 0, None) == status
    assert lib.nvfp4_kv_attention_shared(c, attention(), prefixes(), 0, None, 0, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), INVALID), (dict(q_heads=-1), INVALID), (dict(rows=-1), INVALID), (dict(rot=0), INVALID),
    (dict(rot=-32), INVALID), (dict(rot=160, row_stride=160), INVALID), (dict(row_stride=-4), INVALID),
    (dict(interleaved=2), INVALID), (dict(interleaved=-1), INVALID),
    (dict(tokens=1 << 30), UNSUPPORTED), (dict(q_heads=65537, q_stride=1 << 24, q_out_stride=1 << 24), UNSUPPORTED),
    (dict(rot=16), UNSUPPORTED), (dict(rot=112), UNSUPPORTED), (dict(rot=33), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(tokens=(1 << 30) - 1, q_heads=60000), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(positions=None), INVALID),
    (dict(rotary=None), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID),
    (dict(k=FAKE + 2 * MB + 8), INVALID), (dict(v=FAKE + 3 * MB + 8), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(q_out=FAKE + MB + 8), INVALID), (dict(slots=FAKE + 4 * MB + 4), INVALID),
    (dict(positions=FAKE + 5 * MB + 2), INVALID), (dict(rotary=FAKE + 6 * MB + 8), INVALID),
    (dict(row_stride=130), INVALID), (dict(row_stride=124), INVALID), (dict(k_stride=1020), INVALID),
    (dict(v_stride=1026), INVALID), (dict(q_stride=4092), INVALID), (dict(q_out_stride=4098), INVALID),
    (dict(tokens=0), OK)])
def test_rotary_refusals(lib, change, status):
    assert lib.nvfp4_kv_append_rotary(far_cache(), rotary(**change), 0, None) == status


def test_rotary_options(lib):
    f = lib.nvfp4_kv_append_rotary
    assert f(far_cache(), None, 0, None) == INVALID
    assert f(far_cache(), rotary(), 0x800, None) == INVALID
    assert f(far_cache(), rotary(), 1, None) == INVALID
    assert f(far_cache(), rotary(q=FAKE + 4), 0x400, None) == INVALID  # BF16: 8 bytes


ROW = 4096 * 4  # bytes of a token's queries
# rows of a projection: q 32 heads, k 8, v 8, a stride apart
QKV = dict(q=FAKE, q_stride=6144, k=FAKE + ROW, k_stride=6144, v=FAKE + ROW + 4096, v_stride=6144)


@pytest.mark.parametrize("change", [
    dict(q_out=FAKE + 16), dict(q_out=FAKE - 16), dict(q_out=FAKE + 3 * ROW - 16),
    dict(q_out=FAKE, q_out_stride=4100), dict(q_out=FAKE + 2 * MB), dict(q_out=FAKE + 3 * MB - 2 * ROW),
    dict(q_out=FAKE + 4 * MB - 3 * ROW + 16), dict(q_out=FAKE + 5 * MB), dict(q_out=FAKE + 6 * MB + 99 * 512),
    dict(q_out=FAKE + 14 * MB - ROW), dict(q_out=FAKE + 15 * MB - 2 * ROW), dict(q_out=FAKE + 16 * MB),
    dict(q_out=FAKE + 16 * MB + 9 * 8 * 16 * 144),
    dict(QKV, q_out=FAKE + 16, q_out_stride=6144), dict(QKV, q_out=FAKE + ROW, q_out_stride=6144),
    dict(QKV, q_out=FAKE + 6144 * 4 - ROW + 16, q_out_stride=6144),
    dict(QKV, q_out=FAKE, q_out_stride=6144, k=FAKE + ROW - 16), dict(QKV, q_out=FAKE, q_out_stride=8192)])
def test_rotary_outputs_over_operands(lib, change):
    """Outputs that meet what other threads read are refused."""
    assert lib.nvfp4_kv_append_rotary(far_cache(), rotary(**change), 0, None) == INVALID


def test_rotary_outputs_apart(lib):
    """In place, in the gaps of other rows, and neighbours: as far as the device, which is not there."""
    if torch.cuda.is_available():
        pytest.skip("these addresses are not memory")
    wide = dict(QKV, q_stride=16384, k_stride=16384, v_stride=16384)
    for change in ({}, dict(q_out=FAKE), dict(q_out=FAKE + 3 * ROW), dict(q_out=FAKE - 3 * ROW),
                   dict(q_heads=0, q=None, q_out=None), dict(rows=0, rotary=None), dict(rot=32), dict(interleaved=1),
                   dict(QKV, q_out=FAKE, q_out_stride=6144), dict(tokens=1, q_out=FAKE, q_out_stride=0, q_stride=0),
                   dict(wide, q_out=FAKE + 6144 * 4, q_out_stride=16384),
                   dict(wide, q_out=FAKE - ROW, q_out_stride=16384), dict(rows=1, row_stride=0),
                   dict(q_out=FAKE + 16 * MB + 10 * 8 * 16 * 144)):
        assert lib.nvfp4_kv_append_rotary(far_cache(), rotary(**change), 0, None) == CUDA, change


def test_cross_refusals(lib):
    f = lib.nvfp4_kv_cross_attention
    c = cache()
    for change, status in ((dict(window=4), INVALID), (dict(window=-1), INVALID), (dict(reqs=-1), INVALID),
                           (dict(num_q_heads=33), INVALID), (dict(tokens=1 << 24), UNSUPPORTED),
                           (dict(reqs=16385), UNSUPPORTED), (dict(q=None), INVALID), (dict(seq_len=None), INVALID),
                           (dict(out=FAKE + 8), INVALID), (dict(scale=float("nan")), INVALID),
                           (dict(tokens=0), OK), (dict(reqs=0), OK)):
        assert f(c, attention(**change), 0, None, 0, None) == status
    assert f(c, None, 0, None, 0, None) == INVALID
    assert f(c, attention(), 0x1000, None, 0, None) == INVALID
    assert f(c, attention(), 2, None, 0, None) == UNSUPPORTED  # FP32 on the tcgen05 kernel
    assert f(c, attention(), 0, FAKE + 8, 16, None) == INVALID


def prefixes(**change):
    d = dict(table=FAKE, stride=8, blocks=8, lens=FAKE, start=FAKE, groups=2, scratch=FAKE, size=1 << 30)
    d.update(change)
    return _PREFIXES.pack(*(v or 0 for v in d.values()))


@pytest.mark.parametrize("change,status", [
    (dict(groups=-1), INVALID), (dict(blocks=-1), INVALID), (dict(stride=7), INVALID), (dict(start=None), INVALID),
    (dict(groups=16385), UNSUPPORTED), (dict(blocks=1 << 27, stride=1 << 27), UNSUPPORTED),
    (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(scratch=None), INVALID),
    (dict(lens=FAKE + 2), INVALID), (dict(table=FAKE + 2), INVALID), (dict(start=FAKE + 1), INVALID),
    (dict(scratch=FAKE + 16), INVALID), (dict(size=2 * 32 * (512 + 8)), INVALID), (dict(size=None), INVALID)])
def test_shared_refusals(lib, change, status):
    assert lib.nvfp4_kv_attention_shared(cache(), attention(), prefixes(**change), 0, None, 0, None) == status


def test_shared_refusals_of_the_attention(lib):
    f = lib.nvfp4_kv_attention_shared
    for change, status in ((dict(window=4), INVALID), (dict(reqs=-1), INVALID), (dict(max_q=-1), INVALID),
                           (dict(num_q_heads=8 * 65, q_stride=1 << 20, out_stride=1 << 20), UNSUPPORTED),
                           (dict(num_q_heads=512, tokens=1 << 22, q_stride=1 << 20, out_stride=1 << 20), UNSUPPORTED),
                           (dict(out=None), INVALID), (dict(tokens=0), OK), (dict(reqs=0), OK)):
        assert f(cache(), attention(**change), prefixes(), 0, None, 0, None) == status
    assert f(cache(), attention(), None, 0, None, 0, None) == INVALID
    assert f(cache(), None, prefixes(), 0, None, 0, None) == INVALID
    assert f(cache(), attention(), prefixes(), 0x1000, None, 0, None) == INVALID
    assert f(cache(), attention(), prefixes(), 2, None, 0, None) == UNSUPPORTED
    assert f(cache(), attention(), prefixes(), 0, None, 16, None) == INVALID
    # checks of the prefixes come before "nothing to do"
    assert f(cache(), attention(tokens=0), prefixes(groups=-1), 0, None, 0, None) == INVALID


APART = dict(q=FAKE, out=FAKE + MB, lse=FAKE + 2 * MB)


@pytest.mark.parametrize("change,options", [
    (dict(out=FAKE + 16), 0), (dict(out=FAKE - 16), 0), (dict(out=FAKE + 16), 0xC00), (dict(out=FAKE), 0x400),
    (dict(out=FAKE, out_stride=8192), 0), (dict(out=FAKE + 16 * MB), 0), (dict(out=FAKE + 16 * MB - 16), 0),
    (dict(lse=FAKE + 4), 0), (dict(lse=FAKE + MB + 4), 0), (dict(lse=FAKE + 16 * MB), 0), (dict(lse=FAKE - 4), 0)])
def test_attention_does_not_write_over_what_it_reads(lib, change, options):
    a = attention(**{**APART, **change})
    assert lib.nvfp4_kv_cross_attention(far_cache(), a, options, None, 0, None) == INVALID
    assert lib.nvfp4_kv_attention_shared(far_cache(), a, prefixes(), options, None, 0, None) == INVALID
    assert lib.nvfp4_kv_attention_shared(far_cache(), a, prefixes(groups=0), options, None, 0, None) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls go on to the device's status word")
@pytest.mark.parametrize("change", [dict(), dict(out=FAKE), dict(lse=None), dict(out=FAKE + 48 * 16384),
                                    dict(out=FAKE + 16384, q_stride=8192, out_stride=8192)])
def test_attention_takes_operands_that_do_not_meet(lib, change):
    a = attention(**{**APART, **change})
    assert lib.nvfp4_kv_cross_attention(far_cache(), a, 0, None, 0, None) == CUDA


def test_scratch_size(lib):
    f = lib.nvfp4_kv_shared_scratch_size
    for dim in (64, 128):
        none = f(0, 1, dim)  # the cut items' parts alone
        assert none >= 2 * 64 * 512 * (4 * dim + 8) and none % 16 == 0
        assert f(3, 32, dim) == none + 2 * 3 * 32 * (4 * dim + 8 + 4)
        for tokens in range(1, 9):  # the second pass's half begins on a boundary, whatever the rows
            half = (f(tokens, 7, dim) - 2 * tokens * 7 * 4) // 2
            assert half % 32 == 0 and 0 <= half - none // 2 - tokens * 7 * (4 * dim + 8) < 32
    assert f(-1, 32, 128) == f(3, 0, 128) == f(3, 32, 0) == -INVALID
    assert f(3, 32, 96) == f(1 << 30, 32, 128) == -UNSUPPORTED


def test_calls_want_the_current_device(lib, monkeypatch):
    class Cache:
        _dev, _desc, _workspaces = 0, cache(), {}

    monkeypatch.setattr(nv.kv, "_device", lambda: 1)
    for call in (lambda: nv.kv_append_rotary(Cache, None, None, None, None, None, None),
                 lambda: nv.kv_cross_attention(Cache, None, None, None),
                 lambda: nv.kv_attention_shared(Cache, None, None, None, None, None)):
        with pytest.raises(ValueError, match="current"):
            call()
