"""The paged NVFP4 cache's entry points refuse what they cannot take, on the
host, before any launch.  CPU only: the calls below never reach a kernel."""
import struct

import pytest
import torch

import nvfp4_w4a4_decode_gb300 as nv
from nvfp4_w4a4_decode_gb300 import build as nvbuild
from nvfp4_w4a4_decode_gb300.kv import _CACHE

_ATTENTION = struct.Struct("@PqqPqqPPqqqfqPqP")  # nvfp4_kv_attention_args

FAKE = 1 << 20  # a non-null, aligned value never dereferenced
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return nv.library()


def test_page_bytes(lib):
    assert lib.nvfp4_kv_page_bytes(16, 8, 128) == 8 * 16 * 144
    assert lib.nvfp4_kv_page_bytes(256, 1, 64) == 256 * 72
    for page, heads, dim, status in ((0, 8, 128, INVALID), (16, 0, 128, INVALID), (16, 8, 0, INVALID),
                                     (8, 8, 128, UNSUPPORTED), (48, 8, 128, UNSUPPORTED),
                                     (512, 8, 128, UNSUPPORTED), (16, 8, 96, UNSUPPORTED)):
        assert lib.nvfp4_kv_page_bytes(page, heads, dim) == -status
    with pytest.raises(nv.Nvfp4Error):
        nv.kv_page_bytes(24, 8, 128)


def test_status_bit_is_the_headers():
    assert nv.DEVICE_KV_RANGE == 2 and nv.DEVICE_KV_RANGE & nv.DEVICE_WAIT_TIMEOUT == 0


TABLES = dict(kv_len=FAKE, q_len=FAKE, reqs=4, page=16, free=FAKE, num_free=10, head=FAKE, table=FAKE,
              stride=8, blocks=8, seq=FAKE, start=FAKE, slots=FAKE, pos=FAKE, tokens=4, nxt=FAKE + 64,
              opts=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(reqs=-1), INVALID), (dict(tokens=-1), INVALID), (dict(num_free=-1), INVALID),
    (dict(blocks=-1), INVALID), (dict(stride=7), INVALID), (dict(page=0), INVALID),
    (dict(opts=0x400), INVALID), (dict(page=24), UNSUPPORTED), (dict(reqs=16385), UNSUPPORTED),
    (dict(tokens=1 << 30), UNSUPPORTED), (dict(blocks=1 << 27, stride=1 << 27), UNSUPPORTED),
    (dict(kv_len=None), INVALID), (dict(q_len=None), INVALID), (dict(free=None), INVALID),
    (dict(head=None), INVALID), (dict(nxt=None), INVALID), (dict(nxt=FAKE), INVALID),
    (dict(table=None), INVALID), (dict(seq=None), INVALID), (dict(start=None), INVALID),
    (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(slots=FAKE + 4), INVALID),
    (dict(kv_len=FAKE + 2), INVALID), (dict(table=FAKE + 1), INVALID)])
def test_tables_refusals(lib, change, status):
    assert lib.nvfp4_kv_tables(*{**TABLES, **change}.values()) == status


def cache(**change):
    d = dict(pool=FAKE, k_g=FAKE, v_g=FAKE, num_pages=10, page_stride=8 * 16 * 144, page_size=16,
             num_kv_heads=8, head_dim=128)
    d.update(change)
    return _CACHE.pack(*(v or 0 for v in d.values()))


BAD_CACHES = [(dict(page_size=20), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED),
              (dict(num_kv_heads=0), INVALID), (dict(num_pages=-1), INVALID),
              (dict(page_stride=8 * 16 * 144 - 16), INVALID), (dict(page_stride=8 * 16 * 144 + 8), INVALID),
              (dict(k_g=None), INVALID), (dict(v_g=None), INVALID), (dict(pool=None), INVALID),
              (dict(pool=FAKE + 8), INVALID), (dict(num_pages=1 << 31), INVALID)]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_refusals(lib, change, status):
    c = cache(**change)
    assert lib.nvfp4_kv_append(c, FAKE, 1024, FAKE, 1024, 1, FAKE, 0, None) == status
    a = attention()
    assert lib.nvfp4_kv_attention(c, a, 0, None, 0, None) == status


def test_append_refusals(lib):
    c = cache()
    ref = c
    f = lib.nvfp4_kv_append
    assert f(None, FAKE, 1024, FAKE, 1024, 1, FAKE, 0, None) == INVALID
    assert f(ref, FAKE, 1024, FAKE, 1024, -1, FAKE, 0, None) == INVALID
    assert f(ref, FAKE, 1024, FAKE, 1024, 1 << 30, FAKE, 0, None) == UNSUPPORTED
    assert f(ref, FAKE, 1024, FAKE, 1024, 1, FAKE, 0x800, None) == INVALID
    assert f(ref, FAKE + 8, 1024, FAKE, 1024, 1, FAKE, 0, None) == INVALID      # FP32: 16 bytes
    assert f(ref, FAKE + 4, 1024, FAKE, 1024, 1, FAKE, 0x400, None) == INVALID  # BF16: 8 bytes
    assert f(ref, FAKE, 1020, FAKE, 1024, 2, FAKE, 0, None) == INVALID          # rows overlap
    assert f(ref, FAKE, 1026, FAKE, 1024, 2, FAKE, 0, None) == INVALID          # stride % 4
    assert f(ref, FAKE, 1024, None, 1024, 1, FAKE, 0, None) == INVALID
    assert f(ref, FAKE, 1024, FAKE, 1024, 1, FAKE + 4, 0, None) == INVALID
    assert f(ref, None, 1024, None, 1024, 0, None, 0, None) == OK               # nothing to do


def attention(**change):
    d = dict(q=FAKE, q_stride=4096, num_q_heads=32, block_table=FAKE, table_stride=8, max_blocks=8,
             seq_len=FAKE, q_start=FAKE, reqs=2, tokens=2, max_q=1, scale=0.1, window=0, out=FAKE,
             out_stride=4096, lse=None)
    d.update(change)
    return _ATTENTION.pack(*(v or 0 for v in d.values()))


@pytest.mark.parametrize("change,status", [
    (dict(reqs=-1), INVALID), (dict(tokens=-1), INVALID), (dict(num_q_heads=0), INVALID),
    (dict(num_q_heads=33), INVALID), (dict(num_q_heads=8 * 65, q_stride=1 << 20, out_stride=1 << 20), UNSUPPORTED),
    (dict(max_blocks=-1), INVALID), (dict(table_stride=7), INVALID), (dict(max_q=-1), INVALID),
    (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(tokens=3, q_start=None), INVALID),
    (dict(tokens=1 << 24), UNSUPPORTED), (dict(reqs=16385), UNSUPPORTED),
    (dict(max_blocks=1 << 27, table_stride=1 << 27), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(seq_len=None), INVALID), (dict(block_table=None), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID), (dict(q_stride=4092), INVALID),
    (dict(out_stride=4098), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(tokens=0), OK), (dict(reqs=0), OK)])
def test_attention_refusals(lib, change, status):
    c, a = cache(), attention(**change)
    assert lib.nvfp4_kv_attention(c, a, 0, None, 0, None) == status


def test_attention_options_and_workspace(lib):
    c, a = cache(), attention()
    f, cr, ar = lib.nvfp4_kv_attention, c, a
    assert f(cr, None, 0, None, 0, None) == INVALID
    assert f(cr, ar, 0x1000, None, 0, None) == INVALID     # a flag of other calls
    assert f(cr, ar, 0x77, None, 0, None) == UNSUPPORTED   # no such kernel
    assert f(cr, ar, 0, None, 16, None) == INVALID
    assert f(cr, ar, 0, FAKE + 8, 16, None) == INVALID
    assert lib.nvfp4_kv_attention_workspace_size(128) > lib.nvfp4_kv_attention_workspace_size(64) > 0
    assert lib.nvfp4_kv_attention_workspace_size(0) == -INVALID
    assert lib.nvfp4_kv_attention_workspace_size(96) == -UNSUPPORTED


def test_binding_wants_device_tensors():
    host = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        nv.kv_tables(host, host, host, host, host, page_size=16, tokens=2)
    with pytest.raises(ValueError):
        nv.KVCache(torch.zeros((2, 1, 1152), dtype=torch.uint8), host, host, page_size=16, head_dim=64)


CUDA = 3

# every operand of kv_tables in memory of its own: 4 requests, 10 free pages, 6 rows, a table of 4 x 8 of 12
APART = dict(kv_len=FAKE, q_len=FAKE + 0x100, reqs=4, page=16, free=FAKE + 0x200, num_free=10, head=FAKE + 0x300,
             table=FAKE + 0x400, stride=12, blocks=8, seq=FAKE + 0x600, start=FAKE + 0x700, slots=FAKE + 0x800,
             pos=FAKE + 0x900, tokens=6, nxt=FAKE + 0xA00, opts=0, stream=None)


@pytest.mark.parametrize("change", [
    dict(seq=APART["kv_len"]), dict(seq=APART["kv_len"] + 12), dict(seq=APART["kv_len"] - 12),  # lengths in place
    dict(seq=APART["q_len"]), dict(start=APART["kv_len"] - 16), dict(start=APART["q_len"] + 8),
    dict(slots=APART["kv_len"] - 40), dict(pos=APART["q_len"] + 4), dict(nxt=APART["kv_len"] + 8),
    dict(seq=APART["free"] + 36), dict(pos=APART["free"] - 20), dict(start=APART["head"] - 16),
    dict(nxt=APART["free"]), dict(nxt=APART["head"]), dict(seq=APART["start"]), dict(pos=APART["slots"] + 40),
    dict(nxt=APART["pos"] + 20), dict(nxt=APART["start"] + 16),                  # the last of reqs + 1
    dict(kv_len=APART["table"]), dict(free=APART["table"] - 36), dict(head=APART["table"] + 28),
    dict(seq=APART["table"] + 36), dict(pos=APART["table"] + 24), dict(nxt=APART["table"] + 48 * 3 + 28),
    dict(slots=APART["table"] + 32), dict(kv_len=APART["table"] + 144 - 12)])    # across a gap of 16 bytes
def test_tables_operands_apart(lib, change):
    """A written operand that meets another is refused (kernels would read what others write)."""
    assert lib.nvfp4_kv_tables(*{**APART, **change}.values()) == INVALID


def test_tables_operands_that_touch_only(lib):
    """Neighbours, and vectors in the gap between a table's rows, are as good as apart:
    such calls come as far as the device, which is not there."""
    if torch.cuda.is_available():
        pytest.skip("these addresses are not memory")
    at = FAKE
    for change in ({}, dict(seq=APART["kv_len"] + 16), dict(seq=APART["kv_len"] - 16), dict(nxt=APART["start"] + 20),
                   dict(kv_len=APART["table"] + 32), dict(kv_len=APART["table"] + 144 + 32),
                   dict(head=APART["table"] - 4), dict(nxt=APART["table"] + 176), dict(q_len=APART["kv_len"]),
                   dict(table=at + 0x10000, stride=1 << 24, blocks=1 << 24), dict(reqs=0, seq=FAKE),
                   dict(tokens=0, slots=FAKE, pos=FAKE), dict(blocks=0, seq=APART["table"])):
        assert lib.nvfp4_kv_tables(*{**APART, **change}.values()) == CUDA


def test_calls_want_the_current_device(lib, monkeypatch):
    """Tensors of another device than the current one are refused before anything is launched."""
    class Cache:
        _dev, _desc, _workspaces = 0, cache(), {}

    class Lengths:
        def get_device(self):
            return 0

    monkeypatch.setattr(nv.kv, "_device", lambda: 1)
    for call in (lambda: nv.kv_append(Cache, None, None, None), lambda: nv.kv_attention(Cache, None, None, None),
                 lambda: nv.kv_tables(Lengths(), None, None, None, None, 16, 1),
                 lambda: nv.kv_attention_workspace(64, "cuda:0"), lambda: nv.kv_attention_workspace(64, 0)):
        with pytest.raises(ValueError, match="current"):
            call()
