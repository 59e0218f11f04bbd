"""Plain 64-bit restatement of the paged NVFP4 cache for the tests: pages back
to values by the layout of include/nvfp4_kv.h, attention row by row from its
definition, and the error bounds the kernels are held to."""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def e4m3(b):
    """E4M3 bytes (int64) to float64: bias 7, no infinities, subnormals of 2^-9."""
    s, e, m = b >> 7, (b >> 3) & 15, b & 7
    v = torch.where(e == 0, m.double() * 2.0 ** -9, (8 + m).double() * 2.0 ** (e.double() - 10))
    v = torch.where((b & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(s == 1, -v, v)


def page_values(pages, page_size, dim):
    """uint8 [n, heads, bytes] to (K, V) codes x block scales, float64 [n, heads, page_size, dim]."""
    half, block = page_size * dim // 2, page_size * dim // 16
    parts = pages.long().split((half, half, block, block), -1)

    def values(codes, scales):
        codes = codes.unflatten(-1, (page_size, dim // 2))
        q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        grid = E2M1.to(q.device)
        v = torch.where(q >= 8, -grid[q & 7], grid[q & 7])
        return v * e4m3(scales.unflatten(-1, (page_size, dim // 16))).repeat_interleave(16, -1)

    return values(parts[0], parts[2]), values(parts[1], parts[3])


def request_values(cache, table_row, n):
    """(K, V) float64 [heads, n, dim] of a request's n tokens."""
    pages = table_row[:-(-n // cache.page_size)].long()
    k, v = page_values(cache.pool[pages], cache.page_size, cache.head_dim)
    k, v = (x.transpose(0, 1).flatten(1, 2)[:, :n] for x in (k, v))
    return k * cache.k_g.double(), v * cache.v_g.double()


def attention(cache, q, table, seqs, counts, scale=None, window=0):
    """float64 (out, lse, A, S, B): the definition, sum p |V| / l of each output,
    the largest sum |q| |K| scale of each row, and sum |V| over the keys that a
    row sees (for the bounds)."""
    heads, dim = q.shape[1:]
    group = heads // cache.num_kv_heads
    scale = dim ** -0.5 if scale is None else scale
    q = q.double()
    out, mag, reach = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    big = torch.zeros_like(lse)
    t = 0
    for r, (n, c) in enumerate(zip(seqs, counts)):
        if c and n:
            k, v = request_values(cache, table[r], n)
            k, v = (x.repeat_interleave(group, 0) for x in (k, v))
            qr = q[t:t + c].transpose(0, 1)
            s = qr @ k.transpose(1, 2) * scale
            pos = n - c + torch.arange(c, device=q.device)[:, None]
            key = torch.arange(n, device=q.device)
            hide = key > pos
            if window:
                hide |= key <= pos - window
            s = s.masked_fill(hide, -math.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
            l = p.sum(-1, keepdim=True)
            safe = torch.where(l == 0, 1.0, l)
            out[t:t + c] = (p @ v / safe).transpose(0, 1)
            mag[t:t + c] = (p @ v.abs() / safe).transpose(0, 1)
            reach[t:t + c] = ((~hide).double() @ v.abs()).transpose(0, 1)
            lse[t:t + c] = (m + l.log())[..., 0].T
            big[t:t + c] = (qr.abs() @ k.abs().transpose(1, 2) * abs(scale)).amax(-1).T
        t += c
    return out, lse, mag, big, reach


def check_attention(out, lse, ref, in_dtype):
    """Holds (out, lse) to the reference within what the arithmetic allows.

    A probability's relative error is that of its score: an FP32 sum of D
    exact products (a few 2^-24 of S = sum |q| |K| scale; FP32 queries enter
    with 22 bits, 2^-22 S), one rounded product and difference (2^-23 of it
    each) and the exponential's 2^-22: 2^-19 (1 + S) holds all of it.  BF16
    outputs add the f16 rounding of the probabilities (2^-11) and their own
    (2^-8 of the value), FP32 outputs 2^-22 and the FP32 sums (inside 2^-19).
    f16 is also absolute below its normal range: a probability is stored to
    2^-25, the largest being at least 2^7, so to 2^-32 of the row's largest."""
    want, want_lse, mag, big, reach = ref
    score = 2.0 ** -19 * (1 + big)
    tol = score[..., None] * mag + 2.0 ** -32 * reach
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs() + 2.0 ** -11 * mag
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    worst = (err - tol).max().item()
    assert worst <= 0, f"output off by {err.max().item():.3e}, {worst:.3e} over the bound"
    if lse is not None:
        none = want_lse == -math.inf
        assert torch.equal(lse == -math.inf, none)
        d = torch.where(none, 0.0, lse.double() - want_lse).abs()
        bound = 2.0 * score + 2.0 ** -22 * torch.where(none, 0.0, want_lse).abs()
        assert (d <= bound).all(), f"lse off by {d.max().item():.3e}"
