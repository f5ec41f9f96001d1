"""What the decode-step operators write, they write into the tensor that they were
given: a lazy copy of it (a tensor that shares its memory until one of the two is
written) keeps what it held."""
import pytest

from test_decode_gpu import _gen, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _lazily(torch, t):
    """t, sharing its memory with a copy that has not been made yet; and that copy."""
    return t, torch._lazy_clone(t)


def _setup(torch, dev, heads=2, dim=64):
    gen = _gen(torch, 41)
    pools = [torch.randn((8, 16, heads, dim), generator=gen).bfloat16().to(dev) for _ in range(2)]
    k, v, q = (torch.randn((5, h, dim), generator=gen).bfloat16().to(dev) for h in (heads, heads, 4 * heads))
    table = torch.arange(8, dtype=torch.int32, device=dev).view(1, 8).repeat(5, 1)
    lens = torch.tensor([100, 0, 1, 128, 40], dtype=torch.int32, device=dev)
    return pools, k, v, q, table, lens


def test_append_into_a_lazy_copy(env):  # noqa: F811
    df, torch, dev = env
    pools, k, v, q, _, _ = _setup(torch, dev)
    qo, kept = _lazily(torch, torch.full_like(q, 7.0))
    df.cache_append(df.PagedCache(*pools), k, v, torch.arange(5, device=dev), q=q, q_out=qo)
    assert torch.equal(qo, q) and bool((kept == 7.0).all())
    again, was = _lazily(torch, q.clone())  # in place
    df.cache_append(df.PagedCache(*pools), k, v, torch.arange(5, device=dev), q=again, q_out=again)
    assert torch.equal(again, q) and torch.equal(was, q)


def test_attend_into_a_lazy_copy(env):  # noqa: F811
    df, torch, dev = env
    pools, _, _, q, table, lens = _setup(torch, dev)
    c = df.PagedCache(*pools)
    ws = df.attend_workspace(c, 5, 8, 128, split=32)
    want, wl = torch.empty_like(q), torch.empty((5, 8), device=dev)
    df.attend_paged(want, q, c, table, lens, max_len=128, lse=wl, workspace=ws, split=32)
    out, kept = _lazily(torch, torch.full_like(q, 7.0))
    lse, kept_l = _lazily(torch, torch.full_like(wl, 7.0))
    work, kept_w = _lazily(torch, torch.full_like(ws, 7))
    df.attend_paged(out, q, c, table, lens, max_len=128, lse=lse, workspace=work, split=32)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    for x in (kept, kept_l, kept_w):
        assert bool((x == 7).all())


def test_fold_into_a_lazy_copy(env):  # noqa: F811
    df, torch, dev = env
    outs, lses = torch.randn((3, 9, 64), device=dev), torch.randn((3, 9), device=dev)
    want, wl = torch.empty((9, 64), device=dev), torch.empty(9, device=dev)
    df.fold_softmax(want, outs, lses, lse=wl)
    out, kept = _lazily(torch, torch.full_like(want, 7.0))
    lse, kept_l = _lazily(torch, torch.full_like(wl, 7.0))
    df.fold_softmax(out, outs, lses, lse=lse)
    assert torch.equal(out, want) and torch.equal(lse, wl) and bool((kept == 7.0).all()) and bool((kept_l == 7.0).all())
