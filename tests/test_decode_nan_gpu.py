"""A NaN that a row meets, of any bit pattern, in its query, its keys or its values,
is in its output; and in no other row's or head's."""
import pytest

from test_decode_gpu import NAMES, PAIRS, _cache, _gen, _normal, env  # noqa: F401

pytestmark = pytest.mark.gpu

# NaNs whose set bits lie at the top, at the bottom and with the sign.
PATTERNS = {"f32": ("int32", [0x7FC00000, 0x7F800001, 0x7F80FFFF, -0x7FFFFF, -0x7F0001]), "bf16": ("int16", [0x7FC0, 0x7F81, -0x7F]),
            "f16": ("int16", [0x7E00, 0x7C01, -0x3FF]), "e4m3": ("uint8", [0x7F, 0xFF])}


def _nan(torch, name, i):
    kind, bits = PATTERNS[name]
    x = torch.tensor([bits[i]], dtype=getattr(torch, kind)).view(getattr(torch, NAMES[name]))
    assert bool(torch.isnan(x.float()).all())
    return x[0]


def _set(torch, x, at, value):
    """The bits, as they are: copying a value might quiet a NaN."""
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]
    x.view(kind)[at] = value.view(kind)


def _attend(env, views, q, n):  # noqa: F811
    df, torch, dev = env
    rows = q.shape[0]
    out, lse = torch.empty((rows, q.shape[1], views[1].shape[3]), device=dev, dtype=q.dtype), torch.empty(q.shape[:2], device=dev)
    table = torch.arange(views[0].shape[0], dtype=torch.int32, device=dev).view(rows, -1).contiguous()
    df.attend_paged(out, q.to(dev), df.PagedCache(*views), table, torch.tensor(n, dtype=torch.int32, device=dev), lse=lse)
    return torch.isnan(out).cpu(), torch.isnan(lse).cpu()


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("n", [20, 900])
def test_in_a_query(env, dtype, cache, n):  # noqa: F811
    """Also against keys that an infinity there would give -infinity with."""
    df, torch, dev = env
    for i in range(len(PATTERNS[dtype][1])):
        gen = _gen(torch, 71, n)
        pages = -(-n // 16)
        (k, v), _ = _cache(torch, gen, dev, cache, 2 * pages, 16, 2, 64, 64)
        one = {"e4m3": torch.uint8}.get(cache)
        half = torch.full((1,), -0.5).to(k.dtype)
        (k.view(one) if one else k)[..., 5] = half.view(one)[0] if one else half[0]
        q = _normal(torch, gen, (2, 4, 64), dtype)
        _set(torch, q, (0, 1, 5), _nan(torch, dtype, i))
        out, lse = _attend(env, [k.to(dev), v.to(dev)], q, [n, n])
        assert lse.tolist() == [[False, True, False, False], [False] * 4], i
        assert bool(out[0, 1].all()) and int(out.sum()) == 64, i


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("n,t", [(20, 3), (20, 19), (900, 899), (900, 500), (900, 0)])
def test_in_a_key_or_a_value(env, dtype, cache, n, t):  # noqa: F811
    df, torch, dev = env
    pages = -(-n // 16)
    for i in range(len(PATTERNS[cache][1])):
        gen = _gen(torch, 72, n)
        (k, v), _ = _cache(torch, gen, dev, cache, 2 * pages, 16, 2, 64, 64)
        q = _normal(torch, gen, (2, 4, 64), dtype)
        _set(torch, k, (t // 16, t % 16, 0, 63), _nan(torch, cache, i))
        _set(torch, v, (t // 16, t % 16, 1, 6), _nan(torch, cache, i))
        out, lse = _attend(env, [k.to(dev), v.to(dev)], q, [n, n])
        assert lse.tolist() == [[True, True, False, False], [False] * 4], i
        assert bool(out[0, :2].all()) and bool(out[0, 2:, 6].all()) and int(out.sum()) == 2 * 64 + 2, i
