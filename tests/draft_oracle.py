"""Plain 64-bit forms of the drafted step's operators (CPU), and the error that
their 32-bit computation may have.  Nothing here uses the library.

The tolerances are ``decode_oracle``'s, with what a cap and a bias add to the
error ds of a score s (u = 2^-24):

* s' = cap * tanh(s / cap) has a slope of at most 1, so ds stays; the quotient,
  the hyperbolic tangent and the product add at most 32 u |s'| (the tangent
  itself is held to 24 u relative, its argument's rounding gives at most u, the
  product u, and the rest is room for the second-order terms);
* s' + slope * distance adds 2 u |slope * distance| (the product and, below 2^24,
  an exact distance) and u |s''| for the sum.
"""
import math

import torch

from decode_oracle import U, half_step


def seen_by(n, lens, count, masks, depths, window):
    """[n queries, lens tokens]: what each sees, and the positions' distance (token's less query's)."""
    base = max(lens - count, 0)
    at = lambda j: base + min(max(depths[j], 0), 63)  # noqa: E731
    pos = [t if t < base else at(t - base) for t in range(lens)]
    seen, away = torch.zeros((n, lens), dtype=torch.bool), torch.zeros((n, lens), dtype=torch.float64)
    p = torch.tensor(pos, dtype=torch.float64)
    t = torch.arange(lens)
    for i in range(n):
        bits = (1 << (i + 1)) - 1 if masks is None else masks[i] & (2 ** 64 - 1)
        seen[i] = t < base
        for j in range(min(count, lens - base)):
            seen[i, base + j] = bool(bits >> j & 1)
        away[i] = p - at(i)
        if window:
            seen[i] &= -away[i] < window
    return seen, away


def attend(q, k, v, scale, seen, away, cap, slopes, out_dtype, p_dtype):
    """One row and head: q [n, group, dim], k [tokens, dim], v [tokens, v_dim] in float64, slopes [group] or None.
    Returns out [n, group, v_dim], lse [n, group] and their tolerances.  What a query does not see may hold anything."""
    n, g, dim = q.shape
    if k.shape[0] == 0 or n == 0:
        z = torch.zeros((n, g, v.shape[1]), dtype=torch.float64)
        return z, torch.full((n, g), -math.inf, dtype=torch.float64), z.clone(), torch.zeros((n, g), dtype=torch.float64)
    any_seen = seen.any(0)
    k, v = (torch.where(any_seen[:, None], x, torch.zeros_like(x)) for x in (k, v))
    s = (q.flatten(0, 1) @ k.t()).view(n, g, -1) * scale
    ds = (dim + 4) * U * abs(scale) * (q.abs().flatten(0, 1) @ k.abs().t()).view(n, g, -1)
    if cap:
        s = cap * torch.tanh(s / cap)
        ds = ds + 32 * U * s.abs()
    if slopes is not None:
        b = slopes[None, :, None] * away[:, None]
        s = s + b
        ds = ds + 2 * U * b.abs() + U * s.abs()
    hidden = ~seen[:, None].expand_as(s)
    s = s.masked_fill(hidden, -math.inf)
    ds = torch.where(torch.isfinite(ds) & ~hidden, ds, torch.zeros_like(ds))
    lse = torch.logsumexp(s, -1)
    top = s.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - base)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.zeros((n, g, v.shape[1]), dtype=torch.float64)
    size = torch.zeros_like(out)
    gap = torch.where(torch.isfinite(s), (s - base).abs(), torch.zeros_like(s))
    w = 2 * ds + 2 * U * gap + 2.0 ** -21 + 2 * k.shape[0] * U
    for i in range(n):  # a value that one query does not see is not in its sum, not even times zero
        vi = torch.where(seen[i][:, None], v, torch.zeros_like(v))
        out[i] = p[i] @ vi
        mean = p[i] @ vi.abs()
        size[i] = (p[i] * w[i]) @ vi.abs() + (p[i] * w[i]).sum(-1, keepdim=True) * mean
        if p_dtype is not None:
            size[i] += torch.finfo(p_dtype).eps / 2 * mean
    tol = size + half_step(out.abs() + size, out_dtype)
    lse_tol = (p * w).sum(-1) + ds.amax(-1) + 8 * U * (lse.abs() + base[..., 0].abs() + 1)
    return out, lse, tol, torch.where(torch.isfinite(lse), lse_tol, torch.zeros_like(lse))


def copied(src_cache, dst_cache, src, dst, tokens):
    """Pages [pages, page, heads, dim] after the copies."""
    got = dst_cache.clone()
    for i, (s, d) in enumerate(zip(src, dst)):
        if 0 <= s < src_cache.shape[0] and 0 <= d < dst_cache.shape[0]:
            n = src_cache.shape[1] if tokens is None else min(max(tokens[i], 0), src_cache.shape[1])
            got[d, :n] = src_cache[s, :n]
    return got


def compacted(cache, table, picks, counts, starts, to):
    """The cache [pages, page, heads, dim] after the moves: all reads before any write."""
    got, page = cache.clone(), cache.shape[1]

    def place(tab, x):
        if x < 0 or x >= len(tab) * page:
            return None
        p = tab[x // page]
        return (p, x % page) if 0 <= p < cache.shape[0] else None

    for b in range(len(counts)):
        first = 0 if starts is None else starts[b]
        for i in range(min(max(counts[b], 0), len(picks[b]))):
            pick = picks[b][i]
            if (pick < i if to is None else pick < 0):
                continue
            x, y = place(table[b], first + pick), place(table[b] if to is None else to[b], first + i)
            if x and y:
                got[y] = cache[x]
    return got
