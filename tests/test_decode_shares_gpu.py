"""``attend_paged`` where rows are cut into parts: even shares of all rows' tokens
that begin and end within rows, many rows, and the joins of their parts, against
the 64-bit forms and tolerances of ``decode_oracle.py``."""
import math

import pytest

from test_decode_gpu import PAIRS, _attend_case, _cache, _gen, _normal, env  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(8, 2, 128, 128, 16, "thd"), (15, 3, 84, 84, 7, "thd"), (4, 4, 80, 64, 1, "htd"), (24, 1, 256, 128, 256, "htd"),
          (48, 2, 64, 250, 64, "thd"), (17, 1, 192, 64, 32, "htd"), (6, 6, 17, 19, 3, "thd"), (5, 5, 64, 64, 16, "htd"),
          (36, 2, 32, 32, 48, "thd")]


@pytest.mark.parametrize("q_heads,heads,dim,v_dim,page,order", SHAPES)
@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_shares_of_ragged_rows(env, q_heads, heads, dim, v_dim, page, order, dtype, cache):  # noqa: F811
    _attend_case(env, [700, 0, 1, 333, 2000, 31, 64, 1025], q_heads, heads, dim, v_dim, dtype, cache, page, order)


@pytest.mark.parametrize("q_heads,heads,dim,v_dim,page,order", SHAPES)
@pytest.mark.parametrize("dtype,cache,out", [("bf16", "bf16", "f32"), ("f16", "e4m3", None), ("f32", "f32", None)])
def test_long_steps(env, q_heads, heads, dim, v_dim, page, order, dtype, cache, out):  # noqa: F811
    """More tokens than one step for every wave of the device."""
    _attend_case(env, [9001, 0, 30011, 63, 12345, 1], q_heads, heads, dim, v_dim, dtype, cache, page, order, out=out)


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("window", [257, 300, 1000])
@pytest.mark.parametrize("page", [5, 16])
def test_shares_within_a_window(env, dtype, cache, window, page):  # noqa: F811
    _attend_case(env, [1500, 0, 299, 3001, 40, 301], 6, 2, 64, 64, dtype, cache, page, window=window)


@pytest.mark.parametrize("rows", [63, 64, 65, 130, 300])
@pytest.mark.parametrize("heads", [1, 4])
def test_many_rows(env, rows, heads):  # noqa: F811
    lens = [(i * 7919 + 13) % 600 if i % 5 else 0 for i in range(rows)]
    lens[rows // 2] = 2500
    _attend_case(env, lens, heads, heads, 32, 32, "bf16", "bf16", 16)


def test_all_rows_empty(env):  # noqa: F811
    df, torch, dev = env
    c = df.PagedCache(*(torch.full((3, 16, 2, 64), math.nan, device=dev) for _ in range(2)))
    q = torch.ones((70, 4, 64), device=dev)
    out, lse = torch.full_like(q, 7.0), torch.zeros((70, 4), device=dev)
    table, lens = torch.zeros((70, 100), dtype=torch.int32, device=dev), torch.zeros(70, dtype=torch.int32, device=dev)
    df.attend_paged(out, q, c, table, lens, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_more_rows_than_shares_take(env):  # noqa: F811
    lens = [(i * 31) % 37 for i in range(4100)]
    lens[7], lens[4099] = 300, 290
    _attend_case(env, lens, 2, 1, 16, 16, "f16", "f16", 16)


@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_bad_rows_among_shares(env, dtype, cache):  # noqa: F811
    """As where rows are whole: a page outside the cache or a length past the
    bounds is NaN in its own row, and the rows around it are right."""
    df, torch, dev = env
    gen = _gen(torch, 11)
    (_, _), views = _cache(torch, gen, dev, cache, 50, 16, 2, 64, 64)
    c = df.PagedCache(*views)
    q = _normal(torch, gen, (6, 4, 64), dtype).to(dev)
    table = torch.randint(0, 50, (6, 40), generator=gen, dtype=torch.int32)
    table[1, 39], table[3, 17] = 50, -1
    lens = torch.tensor([640, 640, 600, 300, 641, 1000], dtype=torch.int32)
    out, lse = torch.empty_like(q), torch.empty((6, 4), device=dev)
    df.attend_paged(out, q, c, table.to(dev), lens.to(dev), max_len=900, lse=lse)
    bad = torch.isnan(out).cpu().flatten(1)
    assert bad.all(1).tolist() == bad.any(1).tolist() == [False, True, False, True, True, True]
    assert torch.isnan(lse).cpu().all(1).tolist() == bad.all(1).tolist()
    for b in (0, 2):
        one, l = torch.empty_like(q[:1]), torch.empty((1, 4), device=dev)
        df.attend_paged(one, q[b:b + 1], c, table[b:b + 1].to(dev), lens[b:b + 1].to(dev), lse=l, split=1024)
        eps = torch.finfo(q.dtype).eps
        assert torch.allclose(one[0].float(), out[b].float(), rtol=4 * eps, atol=4 * eps) and torch.allclose(l[0], lse[b], rtol=0, atol=1e-5)


@pytest.mark.parametrize("lens", [[5000, 0, 17, 2999], [70000], [900] * 80])
def test_the_workspace_holds_nothing(env, lens):  # noqa: F811
    """Whatever a workspace holds before a call, and a larger one than needed."""
    df, torch, dev = env
    c, q, table, ln, out, lse = _attend_case(env, lens, 8, 2, 64, 64, "bf16", "bf16", 16)
    for extra in (0, 4096):
        n = df.attend_workspace(c, len(lens), 8, max(lens)).nbytes + extra
        for fill in (0, 255, 127):
            ws = torch.full((n,), fill, dtype=torch.uint8, device=dev)
            o, l = torch.empty_like(q), torch.empty_like(lse)
            for _ in range(2):
                df.attend_paged(o, q, c, table, ln, max_len=max(lens), lse=l, workspace=ws)
                assert torch.equal(o, out) and torch.equal(l, lse)


def test_a_workspace_too_small(env):  # noqa: F811
    df, torch, dev = env
    c = df.PagedCache(*(torch.zeros((64, 16, 2, 64), device=dev) for _ in range(2)))
    q, table = torch.ones((1, 4, 64), device=dev), torch.zeros((1, 64), dtype=torch.int32, device=dev)
    lens = torch.tensor([1000], dtype=torch.int32, device=dev)
    with pytest.raises(df.DetfoldError) as e:
        df.attend_paged(torch.empty_like(q), q, c, table, lens, workspace=torch.empty(64, device=dev))
    assert e.value.rc == df.ESIZE


def test_lengths_change_between_replays(env):  # noqa: F811
    """A captured call follows the lengths and the table, which live on the device."""
    df, torch, dev = env
    c, q, table, ln, out, lse = _attend_case(env, [3000, 800, 17, 2999], 8, 2, 64, 64, "bf16", "bf16", 16)
    ws = df.attend_workspace(c, 4, 8, 3000)
    o, l, lens = torch.empty_like(q), torch.empty_like(lse), ln.clone()
    df.attend_paged(o, q, c, table, lens, max_len=3000, lse=l, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        df.attend_paged(o, q, c, table, lens, max_len=3000, lse=l, workspace=ws)
    for step in (0, 1, 500, 799):
        lens.copy_((ln - step).clamp(min=0))
        graph.replay()
        torch.cuda.synchronize()
        want, wl = torch.empty_like(q), torch.empty_like(lse)
        df.attend_paged(want, q, c, table, lens.clone(), max_len=3000, lse=wl)
        assert torch.equal(o, want) and torch.equal(l, wl), step


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("n", [40, 700])
def test_queries_of_infinity_and_of_the_largest_values(env, dtype, cache, n):  # noqa: F811
    """A score of -infinity everywhere leaves zeros; scores of the type's largest
    values are finite, and alike here."""
    df, torch, dev = env
    gen = _gen(torch, 21, n)
    (_, v), views = _cache(torch, gen, dev, cache, -(-n // 16), 16, 1, 32, 32)
    k = torch.zeros(views[0].shape, device=dev)
    k[..., 0] = 0.5
    c = df.PagedCache(k.to(views[0].dtype), views[1])
    big = torch.finfo(getattr(torch, {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}[dtype])).max
    q = torch.zeros((2, 1, 32), device=dev, dtype=views[0].dtype if dtype == cache else getattr(torch, {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}[dtype]))
    q[0, 0, 0], q[1, 0, 0] = -math.inf, big
    table = torch.arange(-(-n // 16), dtype=torch.int32, device=dev).repeat(2, 1)
    lens = torch.tensor([n, n], dtype=torch.int32, device=dev)
    out, lse = torch.empty_like(q), torch.empty((2, 1), device=dev)
    df.attend_paged(out, q, c, table, lens, lse=lse, scale=0.25)
    assert bool((out[0] == 0).all()) and float(lse[0]) == -math.inf
    # Equal weights of 1: exact but for the sum of n values, the division and the output's rounding.
    seen = v.double().flatten(0, 1)[:n, 0]
    tol = (2 * n * 2.0 ** -24 + 2.0 ** -21) * seen.abs().mean(0) + torch.finfo(q.dtype).eps / 2 * seen.mean(0).abs() + 2.0 ** -24
    assert bool(((out[1, 0].double().cpu() - seen.mean(0)).abs() <= tol).all())
    assert abs(float(lse[1]) / (0.25 * 0.5 * big) - 1) < 1e-3
