"""``attend_paged`` over keys that hold infinities in any place of the head, at
head sizes that fill the kernel's class and at those that do not: a score of
-infinity takes no weight, wherever in the key the infinity stands."""
import math

import pytest

import decode_oracle as oracle
from test_decode_gpu import NAMES, _gen, _normal, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _case(env, dtype, cache, dim, v_dim, at, lens, out=None):  # noqa: F811
    """Every third token's key is -infinity at `at`, where the query is 1: no
    weight.  The others take theirs from finite scores."""
    df, torch, dev = env
    gen = _gen(torch, dtype, cache, dim, v_dim, at)
    page, heads, group = 16, 2, 3
    pages = -(-max(lens) // page)
    k = _normal(torch, gen, (pages, page, heads, dim), cache)
    v = _normal(torch, gen, (pages, page, heads, v_dim), cache)
    k[..., at] = torch.where(torch.arange(pages * page).view(pages, page, 1) % 3 == 1, -math.inf, 0.5)
    q = _normal(torch, gen, (len(lens), heads * group, dim), dtype)
    q[..., at] = 1.0
    c = df.PagedCache(k.to(dev), v.to(dev))
    table = torch.arange(pages, dtype=torch.int32).repeat(len(lens), 1)
    out_t = getattr(torch, NAMES[out or dtype])
    got = torch.empty((len(lens), heads * group, v_dim), device=dev, dtype=out_t)
    lse = torch.empty((len(lens), heads * group), device=dev)
    df.attend_paged(got, q.to(dev), c, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), lse=lse)
    p_type = None if out_t == torch.float32 else out_t
    for b, n in enumerate(lens):
        keep = [t for t in range(n) if t % 3 != 1]
        for h in range(heads):
            i = slice(h * group, (h + 1) * group)
            kd, vd = (x.double().flatten(0, 1)[keep, h] for x in (k, v))
            want, wl, tol, tl = oracle.attend(q[b, i].double(), kd, vd, 1 / math.sqrt(dim), out_t, p_type)
            oracle.close(got[b, i], want, tol, "out of row %d" % b)
            oracle.close(lse[b, i], wl, tl, "lse of row %d" % b)


# Heads that fill their class of 64, 128 or 256, that leave whole or half chunks
# of it, and that a longer value moves to the next class.
HEADS = [(16, 16), (32, 32), (48, 48), (64, 64), (64, 128), (66, 66), (80, 80), (84, 84), (96, 96), (112, 112), (128, 128),
         (128, 192), (160, 160), (192, 192), (193, 64), (224, 128), (240, 240), (256, 256)]


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("dim,v_dim", HEADS)
def test_a_key_of_minus_infinity_takes_no_weight(env, dtype, cache, dim, v_dim):  # noqa: F811
    for at in sorted({0, 1, dim // 2, dim - 8, dim - 4, dim - 2, dim - 1}):
        _case(env, dtype, cache, dim, v_dim, at, [3, 40])


@pytest.mark.parametrize("dtype,cache,out", [("bf16", "bf16", "f32"), ("f16", "f16", "f32"), ("f32", "f32", None)])
@pytest.mark.parametrize("dim", [32, 96, 192])
def test_in_long_rows(env, dtype, cache, out, dim):  # noqa: F811
    _case(env, dtype, cache, dim, dim, dim - 1, [2000, 1, 700], out=out)
