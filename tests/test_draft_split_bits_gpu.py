"""With ``split`` a row's bits are its own: the same in a batch of longer rows, alone,
and whatever ``max_len`` says, through ``attend_tree`` and capped ``attend_paged``."""
import pytest

from test_decode_gpu import _gen, _normal, _cache, _t, env  # noqa: F401

pytestmark = pytest.mark.gpu

LENS = [1000, 3000, 1, 128, 129, 700, 900, 1024, 1025, 1153, 2100, 0]  # 0 to 24 parts of 128 tokens


def _setup(env, dim, v_dim, dtype, cache, drafts, q_heads, heads):  # noqa: F811
    df, torch, dev = env
    gen = _gen(torch, dim, v_dim, dtype, cache, drafts)
    held = [-(-n // 16) for n in LENS]
    _, views = _cache(torch, gen, dev, cache, sum(held) + 1, 16, heads, dim, v_dim)
    table = torch.zeros((len(LENS), max(held)), dtype=torch.int32)
    at = 1
    for b, n in enumerate(held):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    q = _normal(torch, gen, (len(LENS), drafts, q_heads, dim), dtype, 4.0)
    return df.PagedCache(*views), q.to(dev), table.to(dev), torch.tensor(LENS, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("bf16", "bf16"), ("f16", "e4m3")])
@pytest.mark.parametrize("dim,v_dim", [(64, 64), (128, 128), (64, 200)])
@pytest.mark.parametrize("drafts,cap", [(1, 30.0), (3, 0.0), (20, 30.0)])
def test_rows_alone_and_with_other_lengths(env, dtype, cache, dim, v_dim, drafts, cap):  # noqa: F811
    df, torch, dev = env
    c, q, table, lens = _setup(env, dim, v_dim, dtype, cache, drafts, 8, 2)

    def call(rows, **kw):
        out = torch.full((len(rows), drafts, 8, v_dim), 7.0, device=dev)
        lse = torch.full((len(rows), drafts, 8), 7.0, device=dev)
        x = q[rows], table[rows].contiguous(), lens[rows].contiguous()
        if drafts == 1:
            df.attend_paged(out[:, 0], x[0][:, 0], c, x[1], x[2], lse=lse[:, 0], split=128, cap=cap, **kw)
        else:
            df.attend_tree(out, x[0], c, x[1], x[2], lse=lse, split=128, cap=cap, **kw)
        return out, lse
    every = list(range(len(LENS)))
    out, lse = call(every)
    assert bool(torch.isfinite(out).all())
    for most in (3000, 5000, 200000):
        o, l = call(every, max_len=most)  # noqa: E741
        assert torch.equal(o, out) and torch.equal(l, lse), most
    for b, n in enumerate(LENS):
        for most in (n, max(n, 1024), max(n, 1025), 5000):
            o, l = call([b], max_len=most)  # noqa: E741
            assert torch.equal(o[0], out[b]) and torch.equal(l[0], lse[b]), (b, n, most)
    short = [b for b, n in enumerate(LENS) if n <= 1024]
    o, l = call(short, max_len=1024)  # noqa: E741
    assert torch.equal(o, out[short]) and torch.equal(l, lse[short])
