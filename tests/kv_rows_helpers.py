"""Plain 64-bit restatement of attention over keys that are put together from several
places of the paged cache, for the tests (bounds: kv_helpers.check_attention)."""
import math

import torch

from kv_helpers import page_values


def table_values(cache, row, lo, hi):
    """(K, V) float64 [heads, hi - lo, dim] of the tokens [lo, hi) on the pages of a table's row."""
    page, dim = cache.page_size, cache.head_dim
    if hi <= lo:
        return tuple(torch.zeros((cache.num_kv_heads, 0, dim), dtype=torch.float64, device=row.device) for _ in "kv")
    first = lo // page
    at = row[first:-(-hi // page)].tolist()
    assert len(at) == -(-hi // page) - first and all(0 <= p < len(cache.pool) for p in at), "pages of the test's own"
    k, v = page_values(cache.pool[torch.tensor(at, device=row.device)], page, dim)
    k, v = (x.transpose(0, 1).flatten(1, 2)[:, lo - first * page:hi - first * page] for x in (k, v))
    return k * cache.k_g.double(), v * cache.v_g.double()


def attend(q, keys, counts, scale=None, causal=True):
    """float64 (out, lse, mag, big, reach) as of kv_helpers.attention, for requests with these keys
    and values [heads, n, dim] (None: none) and numbers of rows; without `causal` every row sees all."""
    heads, dim = q.shape[1:]
    scale = dim ** -0.5 if scale is None else scale
    q = q.double()
    out, mag, reach = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    big = torch.zeros_like(lse)
    t = 0
    for kv, c in zip(keys, counts):
        if c and kv is not None and kv[0].shape[1]:
            k, v = (x.repeat_interleave(heads // x.shape[0], 0) for x in kv)
            n = k.shape[1]
            qr = q[t:t + c].transpose(0, 1)
            s = qr @ k.transpose(1, 2) * scale
            hide = torch.zeros((c, n), dtype=torch.bool, device=q.device)
            if causal:
                hide = torch.arange(n, device=q.device) > n - c + torch.arange(c, device=q.device)[:, None]
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


def shared_keys(cache, prefix_table, prefix_len, group_start, table, seqs, counts):
    """Each request's keys and values by the definition of shared prefixes."""
    keys = []
    for r, (n, c) in enumerate(zip(seqs, counts)):
        g = next((g for g in range(len(prefix_len)) if group_start[g] <= r < group_start[g + 1]), None)
        p = 0 if g is None else max(prefix_len[g], 0)
        if c == 0:
            keys.append(None)
            continue
        if n - c < p:  # a row inside the prefix: its own pages alone
            p = 0
        k, v = table_values(cache, table[r], p, n)
        if p:
            k0, v0 = table_values(cache, prefix_table[g], 0, p)
            k, v = torch.cat([k0, k], 1), torch.cat([v0, v], 1)
        keys.append((k, v))
    return keys


def rotated(x, positions, rotary, interleaved):
    """x [tokens, heads, dim] float32 with its pairs turned: two products and their sum or
    difference, each rounded to float32 (torch's operations one by one, on the CPU)."""
    x, rows = x.float().cpu(), rotary.cpu()[positions.cpu().long()]
    half = rows.shape[1] // 2
    c, s = rows[:, None, :half], rows[:, None, half:]
    y = x.clone()
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                else (slice(0, half), slice(half, 2 * half)))
    a, b = x[..., one], x[..., two]
    y[..., one] = a * c - b * s
    y[..., two] = b * c + a * s
    return y
