"""Small values: float16 subnormals (below 2^-14) in queries, keys and values, and e4m3
ones (below 2^-6), count as what they are in the attention, the append and the fold."""
import math

import pytest

import decode_oracle as oracle
from test_decode_gpu import NAMES, _gen, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cache,out", [("f16", "f16", None), ("f16", "f16", "f32"), ("f16", "e4m3", None), ("f16", "e4m3", "f32"),
                                             ("bf16", "e4m3", "f32"), ("f32", "e4m3", None)])
@pytest.mark.parametrize("small", ["query", "keys", "values"])
@pytest.mark.parametrize("n", [5, 40, 3000])
def test_attend(env, dtype, cache, out, small, n):  # noqa: F811
    df, torch, dev = env
    gen = _gen(torch, 91, n)
    t, ct = (getattr(torch, NAMES[x]) for x in (dtype, cache))
    tiny = {"query": 2.0 ** -17, "keys": 2.0 ** -17 if cache == "f16" else 2.0 ** -8, "values": 2.0 ** -17 if cache == "f16" else 2.0 ** -8}[small]
    size = {"query": 1.0, "keys": 1.0, "values": 1.0, small: tiny}
    pages = -(-n // 16)
    q = (torch.randn((1, 6, 64), generator=gen) * size["query"]).to(t)
    k, v = ((torch.randn((pages, 16, 2, 64), generator=gen) * size[x]).to(ct) for x in ("keys", "values"))
    scale = 0.125 / (tiny if small != "values" else 1.0)
    ot = getattr(torch, NAMES[out or dtype])
    got, lse = torch.empty((1, 6, 64), device=dev, dtype=ot), torch.empty((1, 6), device=dev)
    df.attend_paged(got, q.to(dev), df.PagedCache(k.to(dev), v.to(dev)), torch.arange(pages, dtype=torch.int32, device=dev).view(1, -1),
                    torch.tensor([n], dtype=torch.int32, device=dev), lse=lse, scale=scale)
    for h in range(2):
        i = slice(3 * h, 3 * h + 3)
        kd, vd = (x.double().flatten(0, 1)[:n, h] for x in (k, v))
        want, wl, tol, tl = oracle.attend(q[0, i].double(), kd, vd, scale, ot, None if ot == torch.float32 else ot)
        oracle.close(got[0, i], want, tol, "out")
        oracle.close(lse[0, i], wl, tl, "lse")
        assert float(want.abs().max()) > 4 * float(tol.max()), "the tolerance would hide what is flushed"


def test_append_and_fold(env):  # noqa: F811
    df, torch, dev = env
    x = torch.arange(1024, dtype=torch.int16).view(torch.float16)  # every subnormal, and its negative
    x = torch.cat([x, -x]).reshape(16, 2, 64)
    c = df.PagedCache(*(torch.zeros((1, 16, 2, 64), device=dev, dtype=torch.float16) for _ in range(2)))
    df.cache_append(c, x.to(dev), x.to(dev), torch.arange(16, device=dev))
    assert torch.equal(c.k[0].cpu(), x) and torch.equal(c.v[0].cpu(), x)
    for t in (torch.float16, torch.float32, torch.bfloat16):
        tiny = torch.finfo(t).smallest_normal
        outs = (torch.randn((3, 50, 64), generator=_gen(torch, 92)) * tiny / 8).to(t)
        out = torch.empty((50, 64), device=dev, dtype=t)
        df.fold_softmax(out, outs.to(dev), torch.zeros((3, 50), device=dev))
        want = outs.double().mean(0)
        # the type's smallest step, and one of binary32's a step of the sum
        tol = torch.full_like(want, oracle.SUB[t] + 4 * 2.0 ** -149) + want.abs() * 2.0 ** -22
        oracle.close(out, want, tol, "fold of %s" % t)
        assert math.isfinite(float(want.abs().max())) and float(want.abs().max()) > 4 * float(tol.max())
