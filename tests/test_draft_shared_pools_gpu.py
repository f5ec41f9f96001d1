"""The compaction, and the copy, on pools whose keys and values, or heads, are one memory:
latent caches, whose values are a view of their keys, and expanded heads.  Lists whose
moves read what others write."""
import random

import pytest

import draft_oracle as oracle
from test_decode_gpu import _gen, _normal, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _bits(torch, x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _views(x, kind, heads, v_dim):
    """Keys and values of a pool [pages, page, heads, dim]."""
    if kind == "same":
        return x, x
    if kind == "first":
        return x, x[..., :v_dim]
    if kind == "last":
        return x, x[..., -v_dim:]
    if kind == "keys within":
        return x[..., 5:5 + v_dim], x
    one = x[:, :, :1].expand(-1, -1, heads, -1)
    return (one, one) if kind == "one head" else (one, one[..., 3:3 + v_dim])


KINDS = ["same", "first", "last", "keys within", "one head", "one head, first"]


@pytest.mark.parametrize("cache", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,dim,v_dim,page,order", [(1, 250, 128, 16, "thd"), (4, 64, 40, 16, "htd"), (8, 128, 96, 7, "thd")])
def test_compact_in_place(env, cache, kind, heads, dim, v_dim, page, order):  # noqa: F811
    df, torch, dev = env
    gen, rng = _gen(torch, cache, kind, heads, dim, page), random.Random(dim)
    batch, n = 6, 600
    held = -(-n // page)
    host = _normal(torch, gen, (batch * held, page, heads, dim), cache)
    pool = host.to(dev) if order == "thd" else host.transpose(1, 2).contiguous().to(dev).transpose(1, 2)
    table = torch.randperm(batch * held, generator=gen).view(batch, held).tolist()
    picks = [list(range(1, n)) + [0], list(range(2, n)) + [0, 0], [min(2 * i + 1, n - 1) for i in range(n)], sorted(rng.sample(range(n), 400)),
             [rng.randrange(n) for _ in range(n)], [0, 2, 3]]
    counts = [len(p) for p in picks]
    picks = [p + [0] * (n - len(p)) for p in picks]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    c = df.PagedCache(*_views(pool, kind, heads, v_dim))
    df.cache_compact(c, i32(table), i32(picks), i32(counts))
    want = host.clone()
    mine = list(_views(host, kind, heads, v_dim))
    wide = mine[1] if kind == "keys within" else mine[0]
    moved = oracle.compacted(_bits(torch, wide.contiguous()), table, picks, counts, None, None)
    if kind.startswith("one head"):
        _bits(torch, want)[:, :, :1] = moved[:, :, :1]
    else:
        _bits(torch, want).copy_(moved)
    assert torch.equal(_bits(torch, pool.cpu().contiguous()), _bits(torch, want.contiguous()))


@pytest.mark.parametrize("kind", KINDS)
def test_copy_and_compact_into_other_pages(env, kind):  # noqa: F811
    df, torch, dev = env
    gen = _gen(torch, kind)
    heads, dim, v_dim, page = 4, 64, 40, 16
    host = _normal(torch, gen, (20, page, heads, dim), "bf16")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    pool = host.to(dev)
    c = df.PagedCache(*_views(pool, kind, heads, v_dim))
    df.cache_copy(c, i32([1, 2, 3]), i32([11, 12, 13]), tokens=i32([16, 5, 1]))
    df.cache_compact(c, i32([[4, 5]]), i32([[31, 3, 3, 17]]), i32([4]), to=i32([[15]]))
    own = slice(0, 1) if kind.startswith("one head") else slice(None)
    want = host.clone()
    for s, d, n in ((1, 11, 16), (2, 12, 5), (3, 13, 1)):
        want[d, :n, own] = host[s, :n, own]
    row = host[4:6].flatten(0, 1)
    want[15, :4, own] = row[[31, 3, 3, 17], own]
    assert torch.equal(pool.cpu(), want)


def test_other_sharing_is_refused(env):  # noqa: F811
    df, torch, dev = env
    x = torch.zeros((6, 16, 4, 64), device=dev, dtype=torch.bfloat16)
    table, picks, counts = (torch.zeros(s, dtype=torch.int32, device=dev) for s in ((1, 2), (1, 4), (1,)))
    for k, v in ((x[..., :40], x[..., 20:]), (x[:, :, :3], x[:, :, 1:]), (x[:5], x[1:]), (x[:, :15], x[:, 1:]),
                 (x[:, :, :1].expand(-1, -1, 4, -1), x), (x[:, :1].expand(-1, 16, -1, -1), torch.zeros_like(x))):
        with pytest.raises(df.DetfoldError) as e:
            df.cache_compact(df.PagedCache(k, v), table, picks, counts)
        assert e.value.rc == df.EOVERLAP
