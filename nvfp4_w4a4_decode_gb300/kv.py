"""Python binding of the paged NVFP4 key/value cache (``include/nvfp4_kv.h``):
``kv_tables``, ``kv_append`` and ``kv_attention`` over a ``KVCache``."""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

__all__ = ["KVCache", "KVTables", "kv_page_bytes", "kv_pool", "kv_tables", "kv_append",
           "kv_attention", "kv_attention_workspace", "nvfp4_kv_tables", "nvfp4_kv_append",
           "nvfp4_kv_attention", "nvfp4_kv_page_bytes", "KERNEL_KV_ROWS", "DEVICE_KV_RANGE"]

KERNEL_KV_ROWS = 1
DEVICE_KV_RANGE = 2

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_u32 = ctypes.c_uint32

SIGNATURES = {
    "nvfp4_kv_page_bytes": ([_i64, _i64, _i64], _i64),
    "nvfp4_kv_tables": ([_p, _p, _i64, _i64, _p, _i64, _p, _p, _i64, _i64, _p, _p, _p, _p, _i64, _p,
                         _u32, _p], ctypes.c_int),
    "nvfp4_kv_append": ([_p, _p, _i64, _p, _i64, _i64, _p, _u32, _p], ctypes.c_int),
    "nvfp4_kv_attention": ([_p, _p, _u32, _p, ctypes.c_size_t, _p], ctypes.c_int),
    "nvfp4_kv_attention_workspace_size": ([_i64], _i64),
}


class _CacheDesc(ctypes.Structure):
    """``nvfp4_kv_cache``."""
    _fields_ = [("pool", _p), ("k_g", _p), ("v_g", _p), ("num_pages", _i64), ("page_stride", _i64),
                ("page_size", _i32), ("num_kv_heads", _i32), ("head_dim", _i32)]


class _AttentionArgs(ctypes.Structure):
    """``nvfp4_kv_attention_args``."""
    _fields_ = [("q", _p), ("q_stride", _i64), ("num_q_heads", _i64), ("block_table", _p),
                ("table_stride", _i64), ("max_blocks", _i64), ("seq_len", _p), ("q_start", _p),
                ("reqs", _i64), ("tokens", _i64), ("max_q", _i64), ("scale", ctypes.c_float),
                ("window", _i64), ("out", _p), ("out_stride", _i64), ("lse", _p)]


from . import (FLAG_PDL, FLAG_X_BF16, FLAG_Y_BF16, KERNEL_AUTO, Nvfp4Error,  # noqa: E402
               library)


def _raise(name, status):
    if status != 0:
        raise Nvfp4Error(name, status)


def _on_device(t, dtype, name, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _vector(t, dtype, name, device, n=None):
    _on_device(t, dtype, name, device)
    if t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be a contiguous vector" + ("" if n is None else f" of {n}"))


def _table(t, rows, device):
    """(pointer, row stride, entries a row) of a block table whose rows are contiguous."""
    _on_device(t, torch.int32, "block_table", device)
    if t.dim() != 2 or t.shape[0] != rows or (t.shape[1] > 1 and t.stride(1) != 1) or \
            (rows > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"block_table must be [{rows}, blocks] with contiguous rows")
    return t.data_ptr(), (t.stride(0) if rows > 1 else t.shape[1]), t.shape[1]


def _heads(t, name, device, dim, dtype=None):
    """Token stride of [tokens, heads, dim] whose token rows are contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype not in ((torch.float32, torch.bfloat16) if dtype is None else (dtype,)):
        raise ValueError(f"{name} must be {dtype or 'float32 or bfloat16'}, got {t.dtype}")
    if t.dim() != 3 or t.shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, heads, {dim}]")
    tokens, heads, _ = t.shape
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != dim) or (tokens > 1 and s[0] < heads * dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return s[0] if tokens > 1 else heads * dim


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
    tensors must stay alive and in place while the cache is used.

    Attention calls on a stream share a zeroed workspace that the cache makes
    at the first of them (one per stream)."""

    def __init__(self, pool, k_g, v_g, page_size: int, head_dim: int):
        _on_device(pool, torch.uint8, "pool")
        _vector(k_g, torch.float32, "k_g", pool.device, 1)
        _vector(v_g, torch.float32, "v_g", pool.device, 1)
        if pool.dim() != 3:
            raise ValueError("pool must be [num_pages, num_kv_heads, bytes]")
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
        self.device = pool.device
        self._desc = _CacheDesc(pool.data_ptr(), k_g.data_ptr(), v_g.data_ptr(), pages,
                                pool.stride(0) if pages > 1 else want, page_size, heads, head_dim)
        self._ref = ctypes.addressof(self._desc)
        self._workspaces = {}

    def _workspace(self, stream: int) -> torch.Tensor:
        ws = self._workspaces.get(stream)
        if ws is None:
            ws = kv_attention_workspace(self.head_dim, self.device)
            # one made while a graph is captured is zeroed by that graph only
            if not torch.cuda.is_current_stream_capturing():
                self._workspaces[stream] = ws
        return ws


def kv_attention_workspace(head_dim: int, device=None) -> torch.Tensor:
    """A zeroed workspace for attention calls that do not overlap in time."""
    n = int(library().nvfp4_kv_attention_workspace_size(head_dim))
    if n < 0:
        raise Nvfp4Error("nvfp4_kv_attention_workspace_size", -n)
    return torch.zeros(n, dtype=torch.uint8,
                       device=device if device is not None else torch.cuda.current_device())


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


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
    the last being the free list's next head.  A free list or table that is
    too short sets DEVICE_KV_RANGE in ``device_status()``."""
    dev = kv_len.device
    _vector(kv_len, torch.int32, "kv_len", None)
    reqs = kv_len.shape[0]
    _vector(q_len, torch.int32, "q_len", dev, reqs)
    _vector(free_pages, torch.int32, "free_pages", dev)
    _vector(free_head, torch.int32, "free_head", dev, 1)
    tp, ts, blocks = _table(block_table, reqs, dev)
    if out is None:
        # one allocation: slots first (8 bytes each), then the int32 vectors
        buf = torch.empty(3 * tokens + 2 * reqs + 2, dtype=torch.int32, device=dev)
        slots, positions, seq, start, head = buf.split((2 * tokens, tokens, reqs, reqs + 1, 1))
        out = KVTables(seq, start, slots.view(torch.int64), positions, head)
    else:
        for t, name, n in ((out.seq_len, "seq_len", reqs), (out.q_start, "q_start", reqs + 1),
                           (out.positions, "positions", tokens), (out.free_head, "free_head", 1)):
            _vector(t, torch.int32, name, dev, n)
        _vector(out.slots, torch.int64, "slots", dev, tokens)
    _raise("nvfp4_kv_tables", library().nvfp4_kv_tables(
        kv_len.data_ptr(), q_len.data_ptr(), reqs, page_size, free_pages.data_ptr(),
        free_pages.shape[0], free_head.data_ptr(), tp, ts, blocks, out.seq_len.data_ptr(),
        out.q_start.data_ptr(), out.slots.data_ptr(), out.positions.data_ptr(), tokens,
        out.free_head.data_ptr(), FLAG_PDL if pdl else 0, _stream(dev)))
    return out


def nvfp4_kv_append(cache: KVCache, k, v, slots, pdl: bool = False) -> None:
    """Quantise keys and values [tokens, num_kv_heads, head_dim] (float32 or
    bfloat16; slices of a projection's rows need no copy) into the cache at
    ``slots`` int64 [tokens] (-1: skipped)."""
    ks = _heads(k, "k", cache.device, cache.head_dim)
    vs = _heads(v, "v", cache.device, cache.head_dim, k.dtype)
    if k.shape != v.shape or k.shape[1] != cache.num_kv_heads:
        raise ValueError(f"k and v must be [tokens, {cache.num_kv_heads}, {cache.head_dim}]")
    _vector(slots, torch.int64, "slots", cache.device, k.shape[0])
    _raise("nvfp4_kv_append", library().nvfp4_kv_append(
        cache._ref, k.data_ptr(), ks, v.data_ptr(), vs, k.shape[0], slots.data_ptr(),
        (FLAG_PDL if pdl else 0) | (FLAG_X_BF16 if k.dtype == torch.bfloat16 else 0),
        _stream(cache.device)))


def nvfp4_kv_attention(cache: KVCache, q, block_table, seq_len, q_start=None, *,
                       max_q: int | None = None, scale: float | None = None, window: int = 0,
                       out=None, out_dtype=None, return_lse: bool = False,
                       kernel: int = KERNEL_AUTO, workspace=None, pdl: bool = False):
    """Causal attention of q [tokens, num_q_heads, head_dim] over the cache.

    ``seq_len`` int32 [reqs]: tokens in the cache, the new ones (already
    appended) included; ``q_start`` int32 [reqs + 1]: each request's first
    query row (None: the same number each).  A request's query rows are its
    last tokens; a row sees its own and earlier positions, the last ``window``
    of them when that is not 0.  ``max_q``: the most rows a request has, if
    known (a hint).  Rows that see nothing get zeros and lse = -inf.
    ``workspace``: one of ``kv_attention_workspace`` (None: the cache's own
    for this stream; False: none, long requests are then not cut).  Output
    float32 or bfloat16 (``out_dtype``, by default q's); with ``return_lse``
    also the natural-log sums [tokens, num_q_heads] float32."""
    dev = cache.device
    qs = _heads(q, "q", dev, cache.head_dim)
    tokens, heads, dim = q.shape
    _vector(seq_len, torch.int32, "seq_len", dev)
    reqs = seq_len.shape[0]
    if q_start is not None:
        _vector(q_start, torch.int32, "q_start", dev, reqs + 1)
    elif reqs and tokens % reqs:
        raise ValueError("without q_start every request has the same number of rows")
    if heads % cache.num_kv_heads:
        raise ValueError(f"{heads} query heads do not share {cache.num_kv_heads} kv heads")
    tp, ts, blocks = _table(block_table, reqs, dev)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=out_dtype or q.dtype, device=dev)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    os_ = _heads(out, "out", dev, dim)
    lse = torch.empty((tokens, heads), dtype=torch.float32, device=dev) if return_lse else None
    stream = _stream(dev)
    if workspace is None:
        workspace = cache._workspace(stream)
    wp = wn = 0
    if workspace is not False:
        _vector(workspace, torch.uint8, "workspace", dev)
        wp, wn = workspace.data_ptr(), workspace.numel()
    if max_q is None:
        max_q = tokens if q_start is not None else (tokens // reqs if reqs else 0)
    args = _AttentionArgs(
        q.data_ptr(), qs, heads, tp, ts, blocks, seq_len.data_ptr(),
        None if q_start is None else q_start.data_ptr(), reqs, tokens, max_q,
        dim ** -0.5 if scale is None else scale, window, out.data_ptr(), os_,
        None if lse is None else lse.data_ptr())
    _raise("nvfp4_kv_attention", library().nvfp4_kv_attention(
        cache._ref, ctypes.addressof(args),
        int(kernel) | (FLAG_PDL if pdl else 0) | (FLAG_X_BF16 if q.dtype == torch.bfloat16 else 0)
        | (FLAG_Y_BF16 if out.dtype == torch.bfloat16 else 0), wp, wn, stream))
    return (out, lse) if return_lse else out


kv_page_bytes = nvfp4_kv_page_bytes
kv_tables = nvfp4_kv_tables
kv_append = nvfp4_kv_append
kv_attention = nvfp4_kv_attention
