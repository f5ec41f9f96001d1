"""``attend_paged`` with scores over the whole range of binary32, whose largest
value is 3.4e38: a score that binary32 holds is not an infinity, whatever units
its exponential is taken in."""
import math

import pytest

from test_decode_gpu import PAIRS, _cache, _gen, _t, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("n", [3, 40, 2500])
@pytest.mark.parametrize("size", [1.5e38, 2.4e38, 3.0e38, 3.38e38])
def test_scores_near_the_largest_value(env, dtype, cache, n, size):  # noqa: F811
    """Rows of equal scores of +size and -size: the mean of the values, exact but for
    the sum of n of them, the division and the output's rounding.  A row of +size
    with every fourth token at -size: those take no weight."""
    df, torch, dev = env
    gen = _gen(torch, 51, n)
    pages = -(-n // 16)
    (_, v), views = _cache(torch, gen, dev, cache, pages, 16, 1, 32, 32)
    sign = torch.ones(pages * 16)
    sign[3::4] = -1.0
    k = torch.zeros((pages, 16, 1, 32))
    k[..., 0], k[..., 31] = 0.5, 0.25 * sign.view(pages, 16, 1)
    c = df.PagedCache(k.to(_t(torch, cache)).to(dev), views[1])
    # 2^14 is exact in every type, and the scale is of the range of the score
    q = torch.zeros((3, 2, 32))
    q[0, :, 0], q[1, :, 0], q[2, :, 31] = 2.0 ** 14, -(2.0 ** 14), 2.0 ** 15
    table = torch.arange(pages, dtype=torch.int32, device=dev).repeat(3, 1)
    lens = torch.full((3,), n, dtype=torch.int32, device=dev)
    out, lse = torch.empty((3, 2, 32), device=dev, dtype=_t(torch, dtype)), torch.empty((3, 2), device=dev)
    scale = size / 2.0 ** 13
    df.attend_paged(out, q.to(_t(torch, dtype)).to(dev), c, table, lens, lse=lse, scale=scale)
    seen = v.double().flatten(0, 1)[:n, 0]
    some = seen[sign[:n] > 0]
    s = float(torch.tensor(scale).float()) * 2.0 ** 13
    for b, (x, want) in enumerate(((seen, s), (seen, -s), (some, s))):
        # 16-bit weights of equal scores are exact: powers of two
        tol = (2 * n * 2.0 ** -24 + 2.0 ** -21) * x.abs().mean(0) + torch.finfo(out.dtype).eps / 2 * x.mean(0).abs() + 2.0 ** -24
        assert bool(((out[b].double().cpu() - x.mean(0)).abs() <= tol).all()), b
        assert bool((lse[b].double().cpu() / want - 1).abs().max() <= 2.0 ** -22), (b, lse[b].tolist())


def test_a_score_past_the_largest_value_is_an_infinity(env):  # noqa: F811
    """-infinity beside others takes no weight; alone, it leaves an empty row."""
    df, torch, dev = env
    gen = _gen(torch, 52)
    (_, v), views = _cache(torch, gen, dev, "f32", 2, 16, 1, 32, 32)
    k = torch.zeros((2, 16, 1, 32), device=dev)
    k[0, :, 0, 0], k[1, :, 0, 0] = -1e20, 1.0
    c = df.PagedCache(k, views[1])
    q = torch.zeros((2, 1, 32), device=dev)
    q[..., 0] = 1e18
    table = torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device=dev)
    lens = torch.tensor([16, 32], dtype=torch.int32, device=dev)
    out, lse = torch.empty((2, 1, 32), device=dev), torch.empty((2, 1), device=dev)
    df.attend_paged(out, q, c, table, lens, lse=lse, scale=8.0)
    assert bool((out[0] == 0).all()) and float(lse[0]) == -math.inf
    assert torch.allclose(out[1, 0].double().cpu(), v[1, :, 0].double().mean(0), rtol=0, atol=1e-6)
    assert abs(float(lse[1]) / 8e18 - 1) < 1e-6
