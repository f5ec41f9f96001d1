"""Calls of the decode-step operators that are too large for one launch, checked
around the border of two: a launch of the attention has at most 2^22 workgroups,
one of the append or the fold at most 2^30 threads."""
import math

import pytest

from test_decode_gpu import _attend_case, env  # noqa: F401

pytestmark = pytest.mark.gpu


def test_attend_many_rows_in_parts(env):  # noqa: F811
    """1024 parts a row, 4096 rows a launch, of the kernel's and of its workspace."""
    lens = [(i * 7919 + 13) % 50 if i % 3 else 0 for i in range(5000)]
    lens[2], lens[4095], lens[4096], lens[4999] = 32768, 3001, 2999, 700
    _attend_case(env, lens, 1, 1, 16, 16, "bf16", "bf16", 16, split=32)


def test_attend_many_whole_rows(env):  # noqa: F811
    """Rows of at most one token, whose output is its value."""
    df, torch, dev = env
    rows, pages = (1 << 22) + 1003, 4099
    v = torch.randn((pages, 1, 1, 16), device=dev).half()
    c = df.PagedCache(torch.randn((pages, 1, 1, 16), device=dev).half(), v)
    table = (torch.arange(rows, device=dev) % pages).int().view(rows, 1)
    lens = (torch.arange(rows, device=dev) % 5 != 3).int()
    out, lse = torch.full((rows, 1, 16), 7.0, device=dev, dtype=torch.float16), torch.empty((rows, 1), device=dev)
    df.attend_paged(out, torch.zeros((rows, 1, 16), device=dev, dtype=torch.float16), c, table, lens, max_len=1, lse=lse)
    want = torch.where(lens[:, None] > 0, v.view(pages, 16)[table[:, 0].long()], torch.zeros((), device=dev, dtype=v.dtype))
    assert torch.equal(out[:, 0], want)
    assert torch.equal(lse[:, 0], torch.where(lens > 0, 0.0, -math.inf))


def test_append_many_tokens(env):  # noqa: F811
    """6 threads a token: 2^30 / 6 tokens a launch.  All tokens have the same key,
    turned by their own positions; all but some have no slot."""
    df, torch, dev = env
    first = (1 << 30) // 6
    tokens = first + 1000
    kept = torch.tensor([0, 1, first - 2, first - 1, first, first + 1, tokens - 1], device=dev)
    slots = torch.full((tokens,), -1, dtype=torch.int64, device=dev)
    slots[kept] = torch.arange(len(kept), device=dev) + 1
    positions = torch.zeros((tokens,), dtype=torch.int64, device=dev)
    positions[kept] = torch.arange(len(kept), device=dev)
    angle = torch.arange(float(len(kept)), device=dev)[:, None] * torch.linspace(1, 0.1, 8, device=dev)
    cos, sin = angle.cos(), angle.sin()
    k, v = torch.randn((1, 1, 16), device=dev), torch.randn((1, 1, 16), device=dev)
    c = df.PagedCache(*(torch.full((3, 16, 1, 16), 7.0, device=dev) for _ in range(2)))
    df.cache_append(c, k.expand(tokens, 1, 16), v.expand(tokens, 1, 16), slots, positions=positions, cos=cos, sin=sin)
    a, b = k[0, 0].double().chunk(2)
    cd, sd = cos.double(), sin.double()
    want = torch.cat([a * cd - b * sd, b * cd + a * sd], 1)
    got = c.k.view(-1, 16)
    # two products and a sum, each half a step of magnitudes up to |a| + |b|
    tol = 3 * 2.0 ** -24 * (a.abs() + b.abs()).repeat(2)
    assert bool(((got[1:len(kept) + 1].double() - want).abs() <= tol).all())
    assert torch.equal(c.v.view(-1, 16)[1:len(kept) + 1], v[0].expand(len(kept), 16))
    for x in (c.k, c.v):
        assert bool((x.view(-1, 16)[0] == 7.0).all()) and bool((x.view(-1, 16)[len(kept) + 1:] == 7.0).all())
    del slots, positions
    torch.cuda.empty_cache()


def test_fold_many_rows(env):  # noqa: F811
    """One thread a row: 2^30 rows a launch.  A single partial is its own mean."""
    df, torch, dev = env
    rows = (1 << 30) + 1000
    outs = torch.arange(rows, device=dev, dtype=torch.float32).view(1, rows, 1)
    lses = torch.zeros((1, rows), device=dev)
    lses[0, ::7] = -math.inf
    out, lse = torch.full((rows, 1), 7.0, device=dev), torch.full((rows,), 7.0, device=dev)
    df.fold_softmax(out, outs, lses, lse=lse)
    want = outs[0, :, 0].clone()
    want[::7] = 0.0
    assert torch.equal(out[:, 0], want) and torch.equal(lse, lses[0])
    del outs, lses, out, lse, want
    torch.cuda.empty_cache()
