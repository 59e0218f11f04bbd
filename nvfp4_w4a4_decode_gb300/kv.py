"""Python binding of the paged NVFP4 key/value cache (``include/nvfp4_kv.h``):
``kv_tables``, ``kv_append`` and ``kv_attention`` over a ``KVCache``.  The checks
of their arguments and their output tensors are made in ``csrc/kv_binding.cpp``."""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import struct
from collections import namedtuple

import torch

__all__ = ["KVCache", "KVTables", "kv_page_bytes", "kv_pool", "kv_tables", "kv_append",
           "kv_attention", "kv_attention_workspace", "nvfp4_kv_tables", "nvfp4_kv_append",
           "nvfp4_kv_attention", "nvfp4_kv_page_bytes", "KERNEL_KV_ROWS", "KERNEL_KV_TILE",
           "DEVICE_KV_RANGE"]

KERNEL_KV_ROWS = 1
KERNEL_KV_TILE = 2
WORKSPACE_ZERO = 4096  # bytes of an attention workspace that start at zero
DEVICE_KV_RANGE = 2

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_u32 = ctypes.c_uint32

SIGNATURES = {
    "nvfp4_kv_page_bytes": ([_i64, _i64, _i64], _i64),
    "nvfp4_kv_tables": ([_p, _p, _i64, _i64, _p, _i64, _p, _p, _i64, _i64, _p, _p, _p, _p, _i64, _p,
                         _u32, _p], ctypes.c_int),
    "nvfp4_kv_append": ([_p, _p, _i64, _p, _i64, _i64, _p, _u32, _p], ctypes.c_int),
    "nvfp4_kv_attention": ([_p, _p, _u32, _p, ctypes.c_size_t, _p], ctypes.c_int),
    "nvfp4_kv_attention_workspace_size": ([_i64], _i64),
}


_CACHE = struct.Struct("@PPPqqiii4x")  # nvfp4_kv_cache


from . import FLAG_PDL, KERNEL_AUTO, Nvfp4Error, library  # noqa: E402
from . import build as _build  # noqa: E402


_calls = None


def _binding():
    """The compiled half of this module, bound to the library (raises if either is not built)."""
    global _calls
    if _calls is None:
        lib = library()
        if not os.path.exists(_build.BINDING):
            raise ImportError(f"{_build.BINDING} is not built; run nvfp4_w4a4_decode_gb300.build.build()")
        loader = importlib.machinery.ExtensionFileLoader("_kv_binding", _build.BINDING)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_file_location("_kv_binding", _build.BINDING, loader=loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.nvfp4_kv_tables, lib.nvfp4_kv_append, lib.nvfp4_kv_attention)), Nvfp4Error)
        _calls = module
    return _calls


def _scale(t, name, dev):
    if t.get_device() != dev or t.dtype is not torch.float32 or t.numel() != 1:
        raise ValueError(f"{name} must be one float32 on CUDA device {dev}")
    return t.data_ptr()


def nvfp4_kv_page_bytes(page_size: int, num_kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of the pool."""
    n = int(library().nvfp4_kv_page_bytes(page_size, num_kv_heads, head_dim))
    if n < 0:
        raise Nvfp4Error("nvfp4_kv_page_bytes", -n)
    return n


def kv_pool(num_pages: int, num_kv_heads: int, head_dim: int, page_size: int = 64,
            device=None) -> torch.Tensor:
    """An uninitialised pool: uint8 [num_pages, num_kv_heads, page_size * 9 * head_dim / 8]."""
    n = nvfp4_kv_page_bytes(page_size, num_kv_heads, head_dim)
    return torch.empty((num_pages, num_kv_heads, n // num_kv_heads), dtype=torch.uint8,
                       device=device if device is not None else torch.cuda.current_device())


class KVCache:
    """The paged NVFP4 cache of one layer over a caller-owned pool.

    ``pool`` is uint8 [num_pages, num_kv_heads, page_size * 9 * head_dim / 8]
    (``kv_pool``) with contiguous pages; the pages themselves may be strided
    (one pool for several layers).  ``k_g`` / ``v_g`` are the tensor scales of
    keys and values ([1] float32, ``global_scale`` of calibration data).  The
    tensors must stay alive and in place while the cache is used, and the
    cache as long as a graph that holds its calls.

    Attention calls on a stream share a workspace that the cache makes at the
    first of them (for each stream used 40 MB at head_dim 128, 20 MB at 64, on 152
    SMs).  A call captured into a graph keeps the workspace of the stream it is
    captured on, where that has one: a graph that may run at the same time as other
    attention calls of that stream takes its own
    (``workspace=kv_attention_workspace(...)``).  Where it has none, the graph holds
    one of its own.  The caches of several layers may be given the same one."""

    def __init__(self, pool, k_g, v_g, page_size: int, head_dim: int):
        if pool.get_device() < 0 or pool.dtype is not torch.uint8 or pool.dim() != 3:
            raise ValueError("pool must be a uint8 CUDA tensor [num_pages, num_kv_heads, bytes]")
        pages, heads, size = pool.shape
        want = nvfp4_kv_page_bytes(page_size, heads, head_dim)
        if size * heads != want:
            raise ValueError(f"pool pages must hold {want} bytes, got {size * heads}")
        if pool.stride(2) != 1 or (heads > 1 and pool.stride(1) != size) or \
                (pages > 1 and pool.stride(0) < want):
            raise ValueError("the pages of the pool must be contiguous")
        self.pool, self.k_g, self.v_g = pool, k_g, v_g
        self.num_pages, self.num_kv_heads = pages, heads
        self.page_size, self.head_dim = int(page_size), int(head_dim)
        self.device, self._dev = pool.device, pool.get_device()
        self._desc = _CACHE.pack(
            pool.data_ptr(), _scale(k_g, "k_g", self._dev), _scale(v_g, "v_g", self._dev), pages,
            pool.stride(0) if pages > 1 else want, page_size, heads, head_dim)
        self._workspaces = {}

    def _workspace(self, stream: int):
        """(address, bytes) of this stream's workspace."""
        ws = self._workspaces.get(stream)
        if ws is None:
            t = kv_attention_workspace(self.head_dim, self.device)
            ws = (t.data_ptr(), t.numel(), t)
            # one made while a graph is captured has its counters zeroed by that graph only
            if not torch.cuda.is_current_stream_capturing():
                self._workspaces[stream] = ws
        return ws


def kv_attention_workspace(head_dim: int, device=None) -> torch.Tensor:
    """A workspace for attention calls that do not overlap in time, on the current
    device (its counters are zero, the rest is whatever the memory held)."""
    if device is not None:
        index = torch.device(device).index
        _current(torch.cuda.current_device() if index is None else index)
    n = int(library().nvfp4_kv_attention_workspace_size(head_dim))
    if n < 0:
        raise Nvfp4Error("nvfp4_kv_attention_workspace_size", -n)
    ws = torch.empty(n, dtype=torch.uint8,
                     device=device if device is not None else torch.cuda.current_device())
    ws[:WORKSPACE_ZERO].zero_()
    return ws


def _raw_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# the same handle without building a Stream object, where torch offers it
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _current(dev: int) -> int:
    """``dev``, which must be the current device: the library launches there, with its
    status word and number of SMs, whatever device the tensors and the stream are of."""
    if _device() != dev:
        raise ValueError(f"the tensors are on CUDA device {dev}, which is not the current one ({_device()})")
    return dev


_OUT = {None: 0, torch.float32: 1, torch.bfloat16: 2}

KVTables = namedtuple("KVTables", "seq_len q_start slots positions free_head")


def nvfp4_kv_tables(kv_len, q_len, free_pages, free_head, block_table, page_size: int, tokens: int,
                    out: KVTables | None = None, pdl: bool = False) -> KVTables:
    """One step's block tables and slot maps from the requests' lengths.

    ``kv_len`` / ``q_len`` int32 [reqs]: tokens held and new tokens;
    ``free_pages`` int32 [n] with its first unused index ``free_head`` int32
    [1]; ``block_table`` int32 [reqs, blocks], whose new entries are filled
    in; ``tokens``: rows of the step (at least ``q_len``'s sum; the rest is
    padding with slot -1).  Returns ``KVTables(seq_len [reqs], q_start
    [reqs + 1], slots [tokens] int64, positions [tokens], free_head [1])``,
    the last being the free list's next head (new tensors, or ``out``, which shares
    no memory with the inputs).  A free list or table that is
    too short sets DEVICE_KV_RANGE in ``device_status()``."""
    dev = kv_len.get_device()
    made = (_calls or _binding()).tables(
        kv_len, q_len, free_pages, free_head, block_table, page_size, tokens, out,
        FLAG_PDL if pdl else 0, _stream(_current(dev)) if dev >= 0 else 0)
    return tuple.__new__(KVTables, made) if out is None else out


def nvfp4_kv_append(cache: KVCache, k, v, slots, pdl: bool = False) -> None:
    """Quantise keys and values [tokens, num_kv_heads, head_dim] (float32 or
    bfloat16; slices of a projection's rows need no copy) into the cache at
    ``slots`` int64 [tokens] (-1: skipped)."""
    (_calls or _binding()).append(cache._desc, cache._dev, k, v, slots, FLAG_PDL if pdl else 0,
                                  _stream(_current(cache._dev)))


def nvfp4_kv_attention(cache: KVCache, q, block_table, seq_len, q_start=None, *,
                       max_q: int | None = None, scale: float | None = None, window: int = 0,
                       out=None, out_dtype=None, return_lse: bool = False,
                       kernel: int = KERNEL_AUTO, workspace=None, pdl: bool = False):
    """Causal attention of q [tokens, num_q_heads, head_dim] over the cache.

    ``seq_len`` int32 [reqs]: tokens in the cache, the new ones (already
    appended) included; ``q_start`` int32 [reqs + 1]: each request's first
    query row (None: the same number each).  A request's query rows are its
    last tokens; a row sees its own and earlier positions, the last ``window``
    of them when that is not 0.  ``max_q``: the most rows a request has (a hint
    for the choice of kernel, worth giving: without it a call with ``q_start`` is
    taken for one request of all rows, right but slow for single tokens).  ``kernel`` forces KERNEL_KV_ROWS or KERNEL_KV_TILE
    (bfloat16 q and output only).  Rows that see nothing get zeros and lse = -inf,
    and so do rows of no request (the padding of a fixed-size batch); in a given
    ``out`` the latter are left as they are.
    ``workspace``: one of ``kv_attention_workspace`` (None: the cache's own
    for this stream; False: none, long requests are then not cut).  Output
    float32 or bfloat16 (``out_dtype``, by default q's); with ``return_lse``
    also the natural-log sums [tokens, num_q_heads] float32."""
    stream = _stream(_current(cache._dev))
    if workspace is None:
        wp, wn, _keep = cache._workspaces.get(stream) or cache._workspace(stream)
    elif workspace is False:
        wp = wn = 0
    else:
        if workspace.get_device() != cache._dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on CUDA device {cache._dev}")
        wp, wn = workspace.data_ptr(), workspace.nbytes
    if out_dtype not in _OUT:
        raise ValueError(f"the output must be float32 or bfloat16, got {out_dtype}")
    return (_calls or _binding()).attention(
        cache._desc, cache._dev, q, block_table, seq_len, q_start, max_q, scale, window, out,
        _OUT[out_dtype], return_lse, kernel | FLAG_PDL if pdl else kernel, wp, wn, stream)


kv_page_bytes = nvfp4_kv_page_bytes
kv_tables = nvfp4_kv_tables
kv_append = nvfp4_kv_append
kv_attention = nvfp4_kv_attention
