"""What no query sees has no part in a result, not even in its last bit: slots behind a
row's end, before a window, and drafted tokens that no mask shows are filled with
zeros, large and infinite values and NaN, and the outputs stay bit for bit."""
import math

import pytest

from test_decode_gpu import PAIRS, _cache, _gen, _normal, _t, env  # noqa: F401

pytestmark = pytest.mark.gpu

LARGE = {"f32": 1e30, "bf16": 1e30, "f16": 6e4, "e4m3": 448.0}


def _bits(torch, x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("drafts,q_heads,heads,dim,page", [(1, 8, 2, 128, 16), (6, 8, 2, 64, 16), (24, 8, 2, 128, 32), (64, 4, 1, 64, 16),
                                                          (5, 3, 1, 84, 7)])
@pytest.mark.parametrize("window", [0, 45])
def test_the_same_bits_whatever_is_hidden(env, dtype, cache, drafts, q_heads, heads, dim, page, window):  # noqa: F811
    df, torch, dev = env
    gen = _gen(torch, dtype, cache, drafts, dim, page, window)
    lens = [drafts, 70, 129, 97, 300]
    lens = [max(n, drafts) for n in lens]
    held = [-(-n // page) for n in lens]
    host, _ = _cache(torch, gen, dev, cache, sum(held) + 2, page, heads, dim, dim)
    table = torch.zeros((len(lens), max(held)), dtype=torch.int32)
    seen = torch.zeros((sum(held) + 2, page), dtype=torch.bool)
    masks = torch.zeros((len(lens), drafts), dtype=torch.int64)
    depths = torch.zeros((len(lens), drafts), dtype=torch.int32)
    at = 1
    for b, n in enumerate(lens):
        table[b, :held[b]] = torch.arange(at, at + held[b], dtype=torch.int32)
        base = n - drafts
        # every third drafted token is hidden from all, itself among them
        shown = [j for j in range(drafts) if (j + b) % 3 or j == 0]
        for i in range(drafts):
            masks[b, i] = sum(1 << j for j in shown if j <= i and j < 63)
            depths[b, i] = i // 2
        t = [t for t in range(base) if not window or base - t < window] + [base + j for j in shown if j < 63]
        if drafts == 1:
            t = [t for t in range(n) if not window or n - 1 - t < window]
        t = torch.tensor(t)
        seen[at + t // page, t % page] = True
        at += held[b]
    ln, tab = torch.tensor(lens, dtype=torch.int32, device=dev), table.to(dev)
    tree = {} if drafts == 1 else dict(masks=masks.to(dev), depths=depths.to(dev))
    for spread, cap in ((0.3, 30.0), (4.0, 5.0), (1.0, 0.0)):  # scores below half the cap, and past it
        q = _normal(torch, gen, (len(lens), drafts, q_heads, dim), dtype, spread).to(dev)
        got = []
        for fill in (None, 0.0, LARGE[cache], -LARGE[cache], math.inf, math.nan):
            if cache == "e4m3" and fill == math.inf:
                continue
            views = []
            for x in host:
                x = x.clone()
                if fill is not None:
                    value = torch.tensor([fill]).to(_t(torch, cache))
                    _bits(torch, x)[~seen] = _bits(torch, value)[0]
                views.append(x.to(dev))
            c = df.PagedCache(*views)
            out, lse = torch.empty((len(lens), drafts, q_heads, dim), device=dev), torch.empty((len(lens), drafts, q_heads), device=dev)
            if drafts == 1:
                df.attend_paged(out[:, 0], q[:, 0], c, tab, ln, lse=lse[:, 0], window=window, cap=cap)
            else:
                df.attend_tree(out, q, c, tab, ln, lse=lse, window=window, cap=cap, **tree)
            narrow = torch.empty_like(q)
            if drafts > 1:
                df.attend_tree(narrow, q, c, tab, ln, window=window, cap=cap, **tree)
            got.append((fill, out, lse, narrow if drafts > 1 else out))
        assert bool(torch.isfinite(got[0][1]).all())
        for fill, *x in got[1:]:
            assert all(torch.equal(y, z) for y, z in zip(x, got[0][1:])), (spread, cap, fill)
