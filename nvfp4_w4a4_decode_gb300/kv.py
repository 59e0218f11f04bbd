"""Python binding of the paged NVFP4 key/value cache (``include/nvfp4_kv.h``):
``kv_tables``, ``kv_append`` and ``kv_attention`` over a ``KVCache``."""
from __future__ import annotations

import ctypes
import struct
from collections import namedtuple

import torch

__all__ = ["KVCache", "KVTables", "kv_page_bytes", "kv_pool", "kv_tables", "kv_append",
           "kv_attention", "kv_attention_workspace", "nvfp4_kv_tables", "nvfp4_kv_append",
           "nvfp4_kv_attention", "nvfp4_kv_page_bytes", "KERNEL_KV_ROWS", "KERNEL_KV_TILE",
           "DEVICE_KV_RANGE"]

KERNEL_KV_ROWS = 1
KERNEL_KV_TILE = 2
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


# nvfp4_kv_cache and nvfp4_kv_attention_args as native struct layouts
_CACHE = struct.Struct("@PPPqqiii4x")
_ATTENTION = struct.Struct("@PqqPqqPPqqqfqPqP")


from . import (FLAG_PDL, FLAG_X_BF16, FLAG_Y_BF16, KERNEL_AUTO, Nvfp4Error,  # noqa: E402
               library)


# The checks run before every call of a decode step, so they read each tensor's
# properties once and in their cheapest form (get_device() is -1 on the host).

def _vector(t, dtype, name, dev, n=-1):
    """Checks a contiguous vector (of n elements) on CUDA device index dev; its address."""
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor (device {dev})")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or not t.is_contiguous() or (n >= 0 and t.numel() != n):
        raise ValueError(f"{name} must be a contiguous vector" + (f" of {n}" if n >= 0 else ""))
    return t.data_ptr()


def _table(t, rows, dev):
    """(address, row stride, entries a row) of a block table whose rows are contiguous."""
    if t.get_device() != dev or t.dtype is not torch.int32:
        raise ValueError(f"block_table must be an int32 tensor on device {dev}")
    if t.dim() != 2:
        raise ValueError(f"block_table must be [{rows}, blocks]")
    n, blocks = t.shape
    step, one = t.stride()
    if n != rows or (blocks > 1 and one != 1) or (rows > 1 and step < blocks):
        raise ValueError(f"block_table must be [{rows}, blocks] with contiguous rows")
    return t.data_ptr(), (step if rows > 1 else blocks), blocks


def _heads(t, name, dev, dim):
    """(tokens, heads, token stride) of [tokens, heads, dim] with contiguous token rows."""
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor (device {dev})")
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.float32:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, {dim}]")
    tokens, heads, d = t.shape
    step, head, one = t.stride()
    if d != dim:
        raise ValueError(f"{name} must be [tokens, heads, {dim}]")
    if one != 1 or (heads > 1 and head != dim) or (tokens > 1 and step < heads * dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return tokens, heads, (step if tokens > 1 else heads * dim)


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
            pool.data_ptr(), _vector(k_g, torch.float32, "k_g", self._dev, 1),
            _vector(v_g, torch.float32, "v_g", self._dev, 1), pages,
            pool.stride(0) if pages > 1 else want, page_size, heads, head_dim)
        self._workspaces = {}

    def _workspace(self, stream: int):
        """(address, bytes) of this stream's workspace."""
        ws = self._workspaces.get(stream)
        if ws is None:
            t = kv_attention_workspace(self.head_dim, self.device)
            ws = (t.data_ptr(), t.numel(), t)
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


def _raw_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# the same handle without building a Stream object, where torch offers it
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


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
    dev, reqs = kv_len.get_device(), kv_len.numel()
    p_len = _vector(kv_len, torch.int32, "kv_len", dev)
    p_new = _vector(q_len, torch.int32, "q_len", dev, reqs)
    p_free = _vector(free_pages, torch.int32, "free_pages", dev)
    p_head = _vector(free_head, torch.int32, "free_head", dev, 1)
    tp, ts, blocks = _table(block_table, reqs, dev)
    if out is None:
        at = kv_len.device
        seq = torch.empty(reqs, dtype=torch.int32, device=at)
        start = torch.empty(reqs + 1, dtype=torch.int32, device=at)
        slots = torch.empty(tokens, dtype=torch.int64, device=at)
        positions = torch.empty(tokens, dtype=torch.int32, device=at)
        head = torch.empty(1, dtype=torch.int32, device=at)
        out = KVTables(seq, start, slots, positions, head)
        outs = (seq.data_ptr(), start.data_ptr(), slots.data_ptr(), positions.data_ptr(), tokens,
                head.data_ptr())
    else:
        outs = (_vector(out.seq_len, torch.int32, "seq_len", dev, reqs),
                _vector(out.q_start, torch.int32, "q_start", dev, reqs + 1),
                _vector(out.slots, torch.int64, "slots", dev, tokens),
                _vector(out.positions, torch.int32, "positions", dev, tokens), tokens,
                _vector(out.free_head, torch.int32, "free_head", dev, 1))
    status = library().nvfp4_kv_tables(p_len, p_new, reqs, page_size, p_free, free_pages.numel(),
                                       p_head, tp, ts, blocks, *outs, FLAG_PDL if pdl else 0,
                                       _stream(dev))
    if status:
        raise Nvfp4Error("nvfp4_kv_tables", status)
    return out


def nvfp4_kv_append(cache: KVCache, k, v, slots, pdl: bool = False) -> None:
    """Quantise keys and values [tokens, num_kv_heads, head_dim] (float32 or
    bfloat16; slices of a projection's rows need no copy) into the cache at
    ``slots`` int64 [tokens] (-1: skipped)."""
    dev = cache._dev
    tokens, heads, ks = _heads(k, "k", dev, cache.head_dim)
    vtokens, vheads, vs = _heads(v, "v", dev, cache.head_dim)
    if heads != cache.num_kv_heads or vheads != heads or vtokens != tokens or k.dtype is not v.dtype:
        raise ValueError(f"k and v must be [tokens, {cache.num_kv_heads}, {cache.head_dim}] of one dtype")
    status = library().nvfp4_kv_append(
        cache._desc, k.data_ptr(), ks, v.data_ptr(), vs, tokens,
        _vector(slots, torch.int64, "slots", dev, tokens),
        (FLAG_PDL if pdl else 0) | (FLAG_X_BF16 if k.dtype is torch.bfloat16 else 0), _stream(dev))
    if status:
        raise Nvfp4Error("nvfp4_kv_append", status)


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
    known (a hint).  ``kernel`` forces KERNEL_KV_ROWS or KERNEL_KV_TILE
    (bfloat16 q and output only).  Rows that see nothing get zeros and lse = -inf.
    ``workspace``: one of ``kv_attention_workspace`` (None: the cache's own
    for this stream; False: none, long requests are then not cut).  Output
    float32 or bfloat16 (``out_dtype``, by default q's); with ``return_lse``
    also the natural-log sums [tokens, num_q_heads] float32."""
    dev, dim = cache._dev, cache.head_dim
    tokens, heads, qs = _heads(q, "q", dev, dim)
    reqs = seq_len.numel()
    p_seq = _vector(seq_len, torch.int32, "seq_len", dev)
    if q_start is not None:
        p_start = _vector(q_start, torch.int32, "q_start", dev, reqs + 1)
    else:
        p_start = 0
        if reqs and tokens % reqs:
            raise ValueError("without q_start every request has the same number of rows")
    if heads % cache.num_kv_heads:
        raise ValueError(f"{heads} query heads do not share {cache.num_kv_heads} kv heads")
    tp, ts, blocks = _table(block_table, reqs, dev)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=out_dtype or q.dtype, device=cache.device)
        os_ = heads * dim
        if out.dtype is not torch.bfloat16 and out.dtype is not torch.float32:
            raise ValueError(f"the output must be float32 or bfloat16, got {out.dtype}")
    else:
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
        os_ = _heads(out, "out", dev, dim)[2]
    lse = torch.empty((tokens, heads), dtype=torch.float32, device=cache.device) if return_lse else None
    stream = _stream(dev)
    if workspace is None:
        wp, wn, _keep = cache._workspace(stream)
    elif workspace is False:
        wp = wn = 0
    else:
        wp, wn = _vector(workspace, torch.uint8, "workspace", dev), workspace.numel()
    if max_q is None:
        max_q = tokens if q_start is not None else (tokens // reqs if reqs else 0)
    args = _ATTENTION.pack(
        q.data_ptr(), qs, heads, tp, ts, blocks, p_seq, p_start, reqs, tokens, max_q,
        dim ** -0.5 if scale is None else scale, window, out.data_ptr(), os_,
        lse.data_ptr() if return_lse else 0)
    status = library().nvfp4_kv_attention(
        cache._desc, args,
        kernel | (FLAG_PDL if pdl else 0) | (FLAG_X_BF16 if q.dtype is torch.bfloat16 else 0)
        | (FLAG_Y_BF16 if out.dtype is torch.bfloat16 else 0), wp, wn, stream)
    if status:
        raise Nvfp4Error("nvfp4_kv_attention", status)
    return (out, lse) if return_lse else out


kv_page_bytes = nvfp4_kv_page_bytes
kv_tables = nvfp4_kv_tables
kv_append = nvfp4_kv_append
kv_attention = nvfp4_kv_attention
