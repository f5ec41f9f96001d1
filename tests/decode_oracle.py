"""Plain 64-bit forms of the decode-step operators (CPU), the error that their
32-bit computation may have, and the inputs the tests share.

Nothing here uses the library.  A tolerance is a bound, element by element:

* a rounding to type t is off by at most half a step, ``eps(t) / 2`` relative
  (half the smallest subnormal below the normal range);
* a binary32 sum of n terms in any order is off by at most ``n * u`` times the
  sum of their magnitudes, u = 2^-24;
* a score s = scale * (q . k) is off by ds <= (dim + 4) u * scale * sum |q_i k_i|
  (the products, the sum, the scale and its product with log2 e), and is
  then taken relative to a maximum with one more rounding; exp's own error is
  below 2^-21 over the whole range that matters.  Every exp(s - m) is thus off
  by the relative error  w = 2 * ds + 2 u |s - m| + 2^-21,  and with p = exp /
  sum the output by  2 * w * sum p |v|  (numerator and denominator);
* the weights may be rounded to the 16-bit type that the matrix units multiply
  (never where the output is float32): eps / 2 * sum p |v| more.
"""
import math

import torch

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
SUB = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, F8: 2.0 ** -10}


def half_step(x, dtype):
    """The largest error of rounding the values x to dtype."""
    return torch.maximum(x.abs() * (torch.finfo(dtype).eps / 2), torch.full_like(x, SUB[dtype]))


def rotate(x, cos, sin, pairs):
    """x [n, heads, dim] in float64 turned by cos, sin [n, half]; and the sum of
    the magnitudes of each value's two products."""
    x = x.clone()
    size = x.abs()
    half = cos.shape[1]
    if half:
        i = torch.arange(half) * 2 if pairs else torch.arange(half)
        j = i + 1 if pairs else i + half
        c, s = cos[:, None], sin[:, None]
        a, b = x[..., i].clone(), x[..., j].clone()
        x[..., i], x[..., j] = a * c - b * s, b * c + a * s
        size[..., i] = (a * c).abs() + (b * s).abs()
        size[..., j] = (b * c).abs() + (a * s).abs()
    return x, size


def stored(x, size, dtype, scale=None):
    """What a cache of `dtype` may hold for the value x (computed in binary32
    with error 2 u size): the value before the last rounding, and the tolerance."""
    tol = 2 * U * size
    if scale is not None:
        x, tol = x / scale[:, None], tol / scale[:, None] + U * (x / scale[:, None]).abs()
    if dtype == F8:
        x = x.clamp(-448, 448)
    return x, tol + half_step(x.abs() + tol, dtype)


def attend(q, k, v, scale, out_dtype, p_dtype):
    """One row and head: q [group, dim], k [n, dim], v [n, v_dim] in float64 (the
    values that the cache stands for).  Returns out, lse and their tolerances."""
    g, n = q.shape[0], k.shape[0]
    if n == 0:
        z = torch.zeros(g, v.shape[1], dtype=torch.float64)
        return z, torch.full((g,), -math.inf, dtype=torch.float64), z.clone(), torch.zeros(g, dtype=torch.float64)
    s = (q @ k.t()) * scale
    lse = torch.logsumexp(s, 1)
    top = s.amax(1, keepdim=True)
    dead = torch.isinf(top) & (top < 0)
    base = torch.where(dead, torch.zeros_like(top), top)
    p = torch.exp(s - base)
    total = p.sum(1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = p @ v
    ds = (q.shape[1] + 4) * U * abs(scale) * (q.abs() @ k.abs().t())
    gap = torch.where(torch.isfinite(s), (s - base).abs(), torch.zeros_like(s))
    ds = torch.where(torch.isfinite(ds), ds, torch.zeros_like(ds))
    w = 2 * ds + 2 * U * gap + 2.0 ** -21 + 2 * n * U
    size = (p * w) @ v.abs() + (p * w).sum(1, keepdim=True) * (p @ v.abs())
    tol = size + (torch.finfo(p_dtype).eps / 2 * (p @ v.abs()) if p_dtype is not None else 0)
    tol = tol + half_step(out.abs() + tol, out_dtype)
    lse_tol = (p * w).sum(1) + ds.amax(1) + 8 * U * (lse.abs() + base[:, 0].abs() + 1)
    return out, lse, tol, torch.where(torch.isfinite(lse), lse_tol, torch.zeros_like(lse))


def fold_softmax(outs, lses, out_dtype):
    """outs [W, rows, dim], lses [W, rows] in float64."""
    lse = torch.logsumexp(lses, 0)
    dead = lses == -math.inf
    a = torch.where(dead, torch.zeros_like(lses), torch.exp(lses - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)))
    o = torch.where(dead[:, :, None], torch.zeros_like(outs), outs)
    out = (a[:, :, None] * o).sum(0)
    w = 2 * U * (lses - lses.amax(0)).abs().nan_to_num(0, 0, 0) + 2.0 ** -21 + (len(lses) + 4) * U
    size = ((a * w)[:, :, None] * o.abs()).sum(0) + (a * w).sum(0)[:, None] * (a[:, :, None] * o.abs()).sum(0)
    tol = size + half_step(out.abs() + size, out_dtype)
    lse_tol = (a * w).sum(0) + 8 * U * (lse.abs().nan_to_num(0, 0, 0) + lses.amax(0).abs().nan_to_num(0, 0, 0) + 1)
    return out, lse, tol, lse_tol


def close(got, want, tol, what):
    """Element by element; NaN and infinities have to be where they are wanted."""
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    odd = ~torch.isfinite(want)
    same = (torch.isnan(got) & torch.isnan(want)) | (got == want)
    assert bool(same[odd].all()), "%s: infinities or NaN differ" % what
    off = torch.where(odd, torch.zeros_like(want), (got - want).abs() - tol.cpu())
    off = torch.where(torch.isnan(off), torch.full_like(off, math.inf), off)
    if off.numel() and float(off.max()) > 0:
        at = int(off.argmax())
        raise AssertionError("%s: %d of %d values are off; worst at %d: got %r want %r tolerance %.3g"
                             % (what, int((off > 0).sum()), off.numel(), at, float(got.flatten()[at]),
                                float(want.flatten()[at]), float(tol.flatten()[at])))
