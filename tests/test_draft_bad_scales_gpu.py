"""A key scale that is no number, or takes the scores past binary32, gives NaN in its
head's results, as in ``attend_paged`` without a cap; and in no other head's."""
import math

import pytest

from test_decode_gpu import _gen, _normal, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 3e38, -3e38], ids=str)
@pytest.mark.parametrize("cap,slopes", [(0.0, False), (30.0, False), (0.0, True), (30.0, True)])
@pytest.mark.parametrize("drafts,dim,n", [(1, 64, 40), (5, 64, 200), (24, 128, 700), (40, 200, 90)])
def test_a_bad_key_scale_is_its_heads_alone(env, dtype, bad, cap, slopes, drafts, dim, n):  # noqa: F811
    df, torch, dev = env
    if drafts == 1 and not cap and not slopes:
        return  # the plain attention, which has tests of its own
    gen = _gen(torch, dtype, drafts, dim, n)
    pages, heads, q_heads = -(-n // 16), 2, 8
    # products of one sign: a scale that is lost would leave all scores equal
    k, v = (_normal(torch, gen, (pages, 16, heads, dim), "e4m3") for _ in range(2))
    k = k.float().abs().add(0.25).to(torch.float8_e4m3fn)
    q = _normal(torch, gen, (1, drafts, q_heads, dim), dtype).abs().to(dev)
    table = torch.arange(pages, dtype=torch.int32, device=dev)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    slope = torch.linspace(0.01, 0.2, q_heads, device=dev) if slopes else None
    args = dict(cap=cap, slopes=slope, scale=2.0 if math.isfinite(bad) else None)
    masks = [(1 << (i + 1)) - 1 for i in range(drafts)]
    got = []
    for scale in (0.5, bad):
        c = df.PagedCache(k.to(dev), v.to(dev), k_scale=torch.tensor([0.25, scale], device=dev), v_scale=torch.tensor([0.5, 2.0], device=dev))
        out, lse = torch.full((1, drafts, q_heads, dim), 7.0, device=dev), torch.full((1, drafts, q_heads), 7.0, device=dev)
        if drafts == 1:
            df.attend_paged(out[:, 0], q[:, 0], c, table, lens, lse=lse[:, 0], **args)
        else:
            df.attend_tree(out, q, c, table, lens, lse=lse, **args, masks=torch.tensor([masks], dtype=torch.int64, device=dev),
                           depths=torch.arange(drafts, dtype=torch.int32, device=dev)[None],
                           counts=torch.tensor([drafts - 1], dtype=torch.int32, device=dev))
        got.append((out, lse))
    (fine, fine_lse), (out, lse) = got
    live = drafts if drafts == 1 else drafts - 1
    assert bool(torch.isfinite(fine).all())
    assert torch.equal(out[:, :, :4], fine[:, :, :4]) and torch.equal(lse[:, :, :4], fine_lse[:, :, :4])
    assert bool(torch.isnan(out[:, :live, 4:]).all()) and bool(torch.isnan(lse[:, :live, 4:]).all())
    assert bool((out[:, live:] == 7.0).all()) and bool((lse[:, live:] == 7.0).all())


def test_rows_without_a_token_stay_empty(env):  # noqa: F811
    df, torch, dev = env
    z = torch.zeros((2, 16, 1, 64), device=dev).to(torch.float8_e4m3fn)
    c = df.PagedCache(z, z.clone(), k_scale=torch.tensor([math.nan], device=dev), v_scale=torch.ones(1, device=dev))
    q, out = torch.ones((1, 3, 2, 64), device=dev), torch.ones((1, 3, 2, 64), device=dev)
    lse = torch.ones((1, 3, 2), device=dev)
    df.attend_tree(out, q, c, torch.zeros((1, 1), dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev), lse=lse,
                   cap=5.0)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
