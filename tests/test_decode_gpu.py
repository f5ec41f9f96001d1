"""The decode-step operators on the device (``cache_append``, ``attend_paged``,
``fold_softmax``) against their 64-bit forms (``decode_oracle.py``, which derives
the tolerances), at the sizes, layouts and masks where they can go wrong."""
import math

import pytest

import decode_oracle as oracle

pytestmark = pytest.mark.gpu

NAMES = {"f32": "float32", "bf16": "bfloat16", "f16": "float16", "e4m3": "float8_e4m3fn"}
PAIRS = [("f32", "f32"), ("f32", "bf16"), ("f32", "e4m3"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f16", "f16"),
         ("f16", "e4m3")]


@pytest.fixture(scope="module")
def env(detfold_lib):
    import torch
    torch.cuda.init()
    return detfold_lib, torch, torch.device("cuda:0")


def _t(torch, name):
    return getattr(torch, NAMES[name])


def _normal(torch, gen, shape, name, spread=1.0):
    return (torch.randn(shape, generator=gen) * spread).to(torch.bfloat16 if name == "e4m3" else _t(torch, name)).to(_t(torch, name))


def _gen(torch, *seed):
    import random
    return torch.Generator().manual_seed(random.Random(repr(seed)).randrange(1 << 40))


def _cache(torch, gen, dev, cache, pages, page, heads, dim, v_dim, order="thd"):
    """Host copies [pages, page, heads, dim] of a filled cache, and its device views."""
    host, views = [], []
    for d in (dim, v_dim):
        x = _normal(torch, gen, (pages, page, heads, d), cache)
        host.append(x)
        if order == "htd":
            views.append(x.transpose(1, 2).contiguous().to(dev).transpose(1, 2))
        elif order == "pair":  # keys and values of a page side by side
            views.append(None)
        else:
            views.append(x.to(dev))
    if order == "pair":
        both = torch.zeros((pages, page, heads, dim + v_dim), dtype=host[0].dtype)
        bits = both.view(torch.uint8)
        size = both.element_size()
        bits[..., :dim * size] = host[0].view(torch.uint8)
        bits[..., dim * size:] = host[1].view(torch.uint8)
        both = both.to(dev)
        views = [both[..., :dim], both[..., dim:]]
    return host, views


def _scales(torch, gen, cache, heads, size):
    if cache != "e4m3":
        return None, None
    s = (torch.rand((2, heads), generator=gen) + 0.5) * size
    return s[0].contiguous(), s[1].contiguous()


def _to(x, dev):
    return None if x is None else x.to(dev)


# --------------------------------------------------------------------------
# cache_append

def _append_case(env, tokens, q_heads, heads, dim, v_dim, dtype, cache, page, rot, pairs, order="thd", idle=(),
                 in_place=False, positions=None, infinite=False):
    df, torch, dev = env
    gen = _gen(torch, tokens, q_heads, heads, dim, v_dim, dtype, cache, page, rot, pairs, order)
    width = q_heads * dim + heads * (dim + v_dim)
    proj = _normal(torch, gen, (tokens, width), dtype)
    if infinite and tokens:
        proj[0, 0], proj[0, -1], proj[-1, 1] = math.inf, -math.inf, math.nan
    ends = [q_heads * dim, heads * dim, heads * v_dim]
    pages = -(-max(tokens, 1) // page) + 3
    host, views = _cache(torch, gen, dev, cache, pages, page, heads, dim, v_dim, order)
    ks, vs = _scales(torch, gen, cache, heads, 0.01)
    slots = torch.randperm(pages * page, generator=gen)[:tokens]
    for i in idle:
        slots[i] = (-1, -5, pages * page, 1 << 40)[i % 4]
    pos = torch.randint(0, 5000, (tokens,), generator=gen) if positions is None else torch.tensor(positions)
    half = rot // 2
    angle = torch.arange(5000, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))
    cos, sin = angle.cos().float(), angle.sin().float()
    c = df.PagedCache(*views, k_scale=_to(ks, dev), v_scale=_to(vs, dev))
    on = proj.to(dev)
    q, k, v = (x.unflatten(1, (-1, d)) if x.shape[1] else None
               for x, d in zip(on.split(ends, dim=1), (dim, dim, v_dim)))
    qo = None if q is None else q if in_place else torch.full((tokens, q_heads, dim), math.nan, device=dev, dtype=on.dtype)
    turn = {} if not rot else dict(positions=pos.to(dev), cos=cos.to(dev), sin=sin.to(dev), pairs=pairs)
    df.cache_append(c, k, v, slots.to(dev), q=q, q_out=qo, **turn)
    torch.cuda.synchronize()

    hq, hk, hv = (x.double().unflatten(1, (-1, d)) if x.shape[1] else None
                  for x, d in zip(proj.split(ends, dim=1), (dim, dim, v_dim)))
    placed = (pos >= 0) & (pos < 5000)
    cs, sn = (torch.where(placed[:, None], x[pos.clamp(0, 4999)].double(), torch.full((), math.nan, dtype=torch.float64))
              for x in (cos, sin))
    if hq is not None:
        want, size = oracle.rotate(hq, cs, sn, pairs)
        oracle.close(qo, want, oracle.stored(want, size, on.dtype)[1], "q_out")
    keep = [i for i in range(tokens) if 0 <= int(slots[i]) < pages * page]
    for at, new, scale, name in ((0, hk, ks, "k"), (1, hv, vs, "v")):
        was = host[at].double().flatten(0, 1)
        want, tol = was.clone(), torch.zeros_like(was)
        x, size = oracle.rotate(new, cs, sn, pairs) if at == 0 else (new, torch.zeros_like(new))
        x, t = oracle.stored(x, size, host[at].dtype, None if scale is None else scale.double())
        for i in keep:
            want[slots[i]], tol[slots[i]] = x[i], t[i]
        if at == 1 and dtype == cache:
            tol = torch.zeros_like(tol)  # a copy
        oracle.close(views[at].cpu().double().flatten(0, 1), want, tol, name)


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("tokens", [1, 2, 67])
@pytest.mark.parametrize("pairs", [False, True])
def test_append_types(env, dtype, cache, tokens, pairs):
    _append_case(env, tokens, 8, 2, 128, 128, dtype, cache, 16, 128, pairs)


@pytest.mark.parametrize("q_heads,heads,dim,v_dim,page,rot,order", [
    (15, 3, 84, 84, 7, 28, "thd"), (4, 4, 80, 64, 1, 40, "htd"), (2, 1, 16, 16, 48, 16, "thd"),
    (16, 8, 256, 128, 256, 64, "pair"), (3, 1, 18, 22, 5, 4, "htd"), (0, 2, 96, 96, 16, 96, "thd"),
    (6, 3, 250, 246, 16, 124, "thd"), (8, 8, 192, 128, 64, 0, "htd"), (2, 2, 17, 19, 3, 0, "thd"),
    (24, 1, 128, 128, 16, 2, "thd"), (5, 1, 66, 33, 9, 66, "pair")])
@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("pairs", [False, True])
def test_append_shapes(env, q_heads, heads, dim, v_dim, page, rot, order, dtype, cache, pairs):
    _append_case(env, 13, q_heads, heads, dim, v_dim, dtype, cache, page, rot, pairs, order, idle=(2, 3, 4, 9))


@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_append_in_place(env, dtype, cache):
    _append_case(env, 9, 8, 2, 64, 64, dtype, cache, 16, 32, False, in_place=True)


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")])
def test_append_infinities_and_bad_positions(env, dtype, cache):
    _append_case(env, 4, 2, 2, 32, 32, dtype, cache, 4, 16, False, infinite=True, positions=[0, -1, 5000, 1 << 40])


def test_append_nothing(env):
    _append_case(env, 0, 8, 2, 64, 64, "bf16", "bf16", 16, 64, False)
    _append_case(env, 5, 8, 2, 64, 64, "bf16", "bf16", 16, 64, False, idle=range(5))


def test_append_e4m3_limits(env):
    """Beyond +-448 the nearest value is the largest; a NaN stays one."""
    df, torch, dev = env
    k = torch.tensor([0.0, -0.0, 448.0, 449.0, 1e30, -1e30, math.inf, -math.inf, math.nan, 2.0 ** -9, 2.0 ** -10,
                      1.5 * 2 ** -10, 464.0, -464.0, 1.0625, 1.1875], device=dev).reshape(1, 1, 16)
    pool = torch.zeros((2, 1, 1, 16), device=dev).to(torch.float8_e4m3fn)
    c = df.PagedCache(pool, pool.clone())
    df.cache_append(c, k, k, torch.tensor([1], device=dev))
    got = c.k.float()[1, 0, 0].cpu().tolist()
    want = [0.0, 0.0, 448.0, 448.0, 448.0, -448.0, 448.0, -448.0, math.nan, 2.0 ** -9, 0.0, 2.0 ** -9, 448.0, -448.0, 1.0, 1.25]
    assert [g if g == g else None for g in got] == [w if w == w else None for w in want]
    assert c.k.float()[0].abs().max() == 0


def test_append_far_slots(env):
    """A cache of more than 2^32 bytes: the last slots are reached, the first stay."""
    df, torch, dev = env
    pages, page, heads, dim = 280000, 16, 4, 128  # 4.6e9 bytes a tensor
    kc = torch.zeros((pages, page, heads, dim), device=dev, dtype=torch.bfloat16)
    c = df.PagedCache(kc, kc)
    k = torch.randn((3, heads, dim), device=dev).bfloat16()
    slots = torch.tensor([pages * page - 1, pages * page - 17, 2 ** 20 + 3], device=dev)
    df.cache_append(c, k, k, slots)
    assert torch.equal(kc.view(-1, heads, dim)[slots], k)
    q = torch.randn((1, 8, dim), device=dev).bfloat16()
    out, table = torch.empty_like(q), torch.tensor([[pages - 1]], device=dev, dtype=torch.int32)
    df.attend_paged(out, q, c, table, torch.tensor([16], device=dev, dtype=torch.int32), window=1)
    want = k[0].repeat_interleave(2, 0)[None]
    assert torch.equal(out, want)  # one token seen: its value itself
    del kc, c
    torch.cuda.empty_cache()


# --------------------------------------------------------------------------
# attend_paged

def _attend_case(env, lens, q_heads, heads, dim, v_dim, dtype, cache, page, order="thd", window=0, out=None,
                 scale=None, split=0, spread=1.0, poison=True, say=None):
    df, torch, dev = env
    gen = _gen(torch, lens, q_heads, heads, dim, v_dim, dtype, cache, page, order, window, out)
    out_t = _t(torch, out or dtype)
    batch, top = len(lens), max(max(lens), 1)
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    host, _ = _cache(torch, gen, torch.device("cpu"), cache, pages, page, heads, dim, v_dim)
    ids = (torch.randperm(pages - 1, generator=gen) + 1).tolist()
    table = torch.full((batch, max(held) + 2), 2 ** 31 - 1, dtype=torch.int32)  # past a row's pages: never read
    seen = []
    nan = 0x7F if cache == "e4m3" else math.nan
    bits = [x.view(torch.uint8) if cache == "e4m3" else x for x in host]
    mask = torch.zeros((pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        mine = [ids.pop() for _ in range(held[b])]
        table[b, :held[b]] = torch.tensor(mine, dtype=torch.int32)
        t = torch.arange(max(0, n - window) if window else 0, n)
        at = (torch.tensor(mine, dtype=torch.long)[t // page], t % page) if n else (t, t)
        seen.append(at)
        mask[at] = True
    if poison:
        for x in bits:
            x[~mask] = nan
    views = [x.transpose(1, 2).contiguous().to(dev).transpose(1, 2) if order == "htd" else x.to(dev) for x in host]
    ks, vs = _scales(torch, gen, cache, heads, 1.0)
    wide = _normal(torch, gen, (batch, q_heads * dim + 8), dtype, spread)
    q = wide.to(dev)[:, :q_heads * dim].unflatten(1, (q_heads, dim))
    c = df.PagedCache(*views, k_scale=_to(ks, dev), v_scale=_to(vs, dev))
    store = torch.full((batch, q_heads, v_dim + 8), 7.0, device=dev, dtype=out_t)
    o, lse = store[..., :v_dim], torch.empty((batch, q_heads), device=dev)
    args = dict(scale=scale, window=window, max_len=top, lse=lse, split=split)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    tab = table.to(dev)
    if say:
        print("case: attend %s" % (say,), flush=True)
    df.attend_paged(o, q, c, tab, ln, **args)
    torch.cuda.synchronize()

    s = 1.0 / math.sqrt(dim) if scale is None else scale
    g = q_heads // heads
    p_type = None if out_t == torch.float32 else out_t
    qd = wide[:, :q_heads * dim].unflatten(1, (q_heads, dim)).double()
    kd, vd = (x.double() * (1.0 if z is None else z.double()[:, None]) for x, z in zip(host, (ks, vs)))
    want = torch.zeros((batch, q_heads, v_dim), dtype=torch.float64)
    tol, wl, tl = torch.zeros_like(want), torch.zeros((batch, q_heads), dtype=torch.float64), torch.zeros((batch, q_heads), dtype=torch.float64)
    for b in range(batch):
        for h in range(heads):
            i = slice(h * g, (h + 1) * g)
            want[b, i], wl[b, i], tol[b, i], tl[b, i] = oracle.attend(
                qd[b, i], kd[seen[b]][:, h], vd[seen[b]][:, h], s, out_t, p_type)
    oracle.close(o, want, tol, "out")
    oracle.close(lse, wl, tl, "lse")
    assert bool((store[..., v_dim:] == 7.0).all()), "written past the head"
    first = o.clone(), lse.clone()
    for _ in range(2):
        store.zero_()
        df.attend_paged(o, q, c, tab, ln, **args)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1]), "two calls differ"
    return c, q, tab, ln, o, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500]


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("out", [None, "f32"])
@pytest.mark.parametrize("order", ["thd", "htd"])
def test_attend_types(env, dtype, cache, out, order):
    _attend_case(env, LENS, 8, 2, 128, 128, dtype, cache, 16, order, out=out)


@pytest.mark.parametrize("q_heads,heads,dim,v_dim,page,order", [
    (15, 3, 84, 84, 7, "thd"), (4, 4, 80, 64, 1, "htd"), (16, 1, 16, 16, 48, "thd"), (24, 1, 256, 128, 256, "htd"),
    (3, 3, 18, 22, 5, "htd"), (96, 2, 64, 256, 64, "thd"), (7, 1, 250, 246, 16, "thd"), (17, 1, 192, 64, 32, "htd"),
    (2, 2, 17, 19, 3, "thd"), (33, 1, 96, 96, 128, "thd"), (12, 12, 40, 132, 16, "thd"), (5, 1, 136, 72, 9, "htd")])
@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_attend_shapes(env, q_heads, heads, dim, v_dim, page, order, dtype, cache):
    _attend_case(env, [0, 1, 30, 65, 200], q_heads, heads, dim, v_dim, dtype, cache, page, order)


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("window", [1, 3, 16, 33, 100, 400, 5000])
def test_attend_window(env, dtype, cache, window):
    _attend_case(env, [0, 1, 40, 64, 99, 100, 101, 417], 6, 2, 64, 64, dtype, cache, 16, window=window)


@pytest.mark.parametrize("dtype,cache,lens", [("bf16", "bf16", [5003]), ("f16", "e4m3", [20011, 3, 0, 7777]),
                                              ("f32", "f32", [4097, 1]), ("bf16", "e4m3", [70001])])
@pytest.mark.parametrize("split", [0, 32, 256, 4096])
def test_attend_long_and_split(env, dtype, cache, lens, split):
    _attend_case(env, lens, 8, 2, 128, 128, dtype, cache, 16, split=split)


@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_attend_sharp_and_flat(env, dtype, cache):
    """Scores far apart (one token takes all), and all alike (scale 0)."""
    _attend_case(env, [1, 50, 300], 4, 1, 64, 64, dtype, cache, 16, spread=30.0)
    _attend_case(env, [1, 50, 300], 4, 1, 64, 64, dtype, cache, 16, scale=0.0)
    _attend_case(env, [1, 50, 300], 4, 1, 64, 64, dtype, cache, 16, scale=-0.3)


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_attend_lowest_scores(env, dtype, cache):
    """Keys of the type's lowest value: scores of about -1e38 and -infinity take
    no weight beside others, and leave zeros where there is nothing else."""
    df, torch, dev = env
    t = _t(torch, cache)
    k = torch.zeros((3, 16, 1, 64), dtype=t)
    v = torch.randn((3, 16, 1, 64), generator=_gen(torch, 1)).to(t)
    k[0] = torch.finfo(t).min
    k[1, :, :, 0] = torch.finfo(t).min
    k[2, :, :, 0] = -math.inf
    q = torch.zeros((4, 2, 64), dtype=_t(torch, dtype))
    q[..., 0] = 1.0
    q[0] = 1.0  # 64 times the lowest value: -infinity
    table = torch.tensor([[0, 0], [1, 1], [2, 2], [2, 1]], dtype=torch.int32)
    lens = torch.tensor([20, 20, 20, 20], dtype=torch.int32)
    c = df.PagedCache(k.to(dev), v.to(dev))
    out, lse = torch.empty_like(q, device=dev), torch.empty((4, 2), device=dev)
    df.attend_paged(out, q.to(dev), c, table.to(dev), lens.to(dev), lse=lse, scale=0.25)
    low = 0.25 * float(torch.finfo(t).min)
    vd = v.double()[:, :, 0]
    means = [torch.zeros(64, dtype=torch.float64), torch.cat([vd[1], vd[1, :4]]).mean(0), torch.zeros(64, dtype=torch.float64),
             vd[1, :4].mean(0)]
    want = torch.stack(means)[:, None].expand(4, 2, 64)
    tol = torch.full_like(want, 4 * torch.finfo(_t(torch, dtype)).eps * 4)
    oracle.close(out, want, tol, "out")
    got = lse.double().cpu()
    assert bool((got[[0, 2]] == -math.inf).all())
    assert torch.allclose(got[[1, 3]], torch.full((2, 2), low, dtype=torch.float64), rtol=1e-6)


def test_attend_nan_where_it_is_seen(env):
    """A NaN key or value that a row sees is that row's and head's alone."""
    df, torch, dev = env
    gen = _gen(torch, 2)
    k, v = (torch.randn((4, 16, 2, 64), generator=gen).bfloat16() for _ in range(2))
    k[1, 3, 0, 5] = math.nan
    v[2, 4, 1, 6] = math.nan
    c = df.PagedCache(k.to(dev), v.to(dev))
    q = torch.randn((3, 4, 64), generator=gen).bfloat16().to(dev)
    table = torch.tensor([[1, 0], [2, 0], [3, 0]], dtype=torch.int32, device=dev)
    out, lse = torch.empty_like(q), torch.empty((3, 4), device=dev)
    df.attend_paged(out, q, c, table, torch.tensor([20, 20, 20], dtype=torch.int32, device=dev), lse=lse)
    bad = torch.isnan(out).cpu()
    assert bool(bad[0, :2].all()) and not bool(bad[0, 2:].any())
    assert not bool(bad[1, :2].any()) and bool(bad[1, 2:, 6].all()) and int(bad[1].sum()) == 2
    assert not bool(bad[2].any())
    assert torch.isnan(lse).cpu().tolist() == [[True, True, False, False], [False] * 4, [False] * 4]


@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_attend_bad_rows_are_nan(env, dtype, cache):
    """A page outside the cache, a length past max_len or the table: NaN in that
    row alone, and nothing read out of range; a negative length is an empty row."""
    df, torch, dev = env
    gen = _gen(torch, 3)
    (_, _), views = _cache(torch, gen, dev, cache, 5, 16, 2, 64, 64)
    c = df.PagedCache(*views)
    q = _normal(torch, gen, (8, 4, 64), dtype).to(dev)
    good = [1, 2, 3, 4]
    table = torch.tensor([good, [1, 5, 3, 4], [1, 2, -1, 4], [1, 2, 3, 2 ** 31 - 1], good, good, good, good],
                         dtype=torch.int32, device=dev)
    lens = torch.tensor([64, 64, 64, 64, 65, 2 ** 31 - 1, -3, 50], dtype=torch.int32, device=dev)
    for split in (0, 32):
        out, lse = torch.empty_like(q), torch.empty((8, 4), device=dev)
        df.attend_paged(out, q, c, table, lens, max_len=100, lse=lse, split=split)
        bad = torch.isnan(out).cpu().flatten(1)
        assert bad.all(1).tolist() == [False, True, True, True, True, True, False, False]
        assert bad.any(1).tolist() == [False, True, True, True, True, True, False, False]
        assert bool((out[6] == 0).all()) and bool((lse[6] == -math.inf).all())
        assert torch.isnan(lse).cpu().all(1).tolist() == bad.all(1).tolist()
        df.attend_paged(out, q, c, table, lens, max_len=49, lse=lse, split=split)
        assert torch.isnan(out).cpu().flatten(1).all(1).tolist() == [True] * 6 + [False, True]


def test_attend_rows_alone_give_the_same_bits(env):
    """With a split of the caller's, a row's bits do not depend on the batch."""
    df, torch, dev = env
    c, q, table, lens, out, lse = _attend_case(env, [900, 33, 2000, 1], 8, 2, 128, 128, "bf16", "bf16", 16, split=128)
    for b in range(4):
        o, l = torch.empty_like(q[:1]), torch.empty((1, 8), device=dev)
        df.attend_paged(o, q[b:b + 1], c, table[b:b + 1], lens[b:b + 1], lse=l, split=128)
        assert torch.equal(o[0], out[b]) and torch.equal(l[0], lse[b])


def test_attend_nothing(env):
    df, torch, dev = env
    _attend_case(env, [0, 0], 4, 2, 64, 64, "bf16", "bf16", 16)
    c = df.PagedCache(*(torch.zeros((1, 16, 2, 64), device=dev) for _ in range(2)))
    q = torch.zeros((0, 4, 64), device=dev)
    i = torch.zeros((0,), dtype=torch.int32, device=dev)
    df.attend_paged(q.clone(), q, c, i.view(0, 1), i)
    q, i = torch.ones((2, 4, 64), device=dev), torch.zeros((2,), dtype=torch.int32, device=dev)
    df.attend_paged(out := torch.ones_like(q), q, c, i.view(2, 1)[:, :0], i)  # a table of no pages
    assert bool((out == 0).all())


def test_attend_streams_and_graph(env):
    """On a stream of the caller's, and captured: every replay gives the eager bits."""
    df, torch, dev = env
    c, q, table, lens, out, lse = _attend_case(env, [3000, 0, 17, 2999], 8, 2, 128, 128, "bf16", "bf16", 16)
    want = out.clone(), lse.clone()
    ws = df.attend_workspace(c, 4, 8, 3000)
    o, l = torch.empty_like(want[0]), torch.empty_like(want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        df.attend_paged(o, q, c, table, lens, max_len=3000, lse=l, workspace=ws)
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    graph = torch.cuda.CUDAGraph()
    k = torch.randn((4, 2, 128), device=dev).bfloat16()
    slots = torch.tensor([5, -1, -1, 9], device=dev)  # page 0 is no row's
    with torch.cuda.graph(graph):
        df.cache_append(c, k, k, slots)
        df.attend_paged(o, q, c, table, lens, max_len=3000, lse=l, workspace=ws)
    for _ in range(4):
        o.zero_(), l.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
        df.attend_paged(o, q, c, table, lens, max_len=3000, lse=l, workspace=ws)  # eager work between
        torch.cuda.synchronize()


# --------------------------------------------------------------------------
# fold_softmax

def _fold_case(env, W, shape, dim, dtype, empty=0.0, pad=0, spread=3.0):
    df, torch, dev = env
    gen = _gen(torch, W, shape, dim, dtype, empty, pad)
    n = math.prod(shape)
    outs = _normal(torch, gen, (W, n, dim), dtype)
    lses = torch.randn((W, n), generator=gen) * spread + 6
    if empty:
        lses[torch.rand((W, n), generator=gen) < empty] = -math.inf
        if n > 1:
            lses[:, n // 2] = -math.inf
        outs[lses == -math.inf] = math.nan
    big, small = torch.zeros((W, n * dim + pad), dtype=outs.dtype), torch.zeros((W, n + pad))
    big[:, :n * dim], small[:, :n] = outs.flatten(1), lses
    big, small = big.to(dev), small.to(dev)
    o, l = big[:, :n * dim].view(W, *shape, dim), small[:, :n].view(W, *shape)
    out, lse = torch.empty((*shape, dim), device=dev, dtype=outs.dtype), torch.empty(shape, device=dev)
    df.fold_softmax(out, o, l, lse=lse)
    want, wl, tol, tl = oracle.fold_softmax(outs.double(), lses.double(), outs.dtype)
    oracle.close(out.flatten(0, -2), want, tol, "out")
    oracle.close(lse.flatten(), wl, tl, "lse")
    again = torch.empty_like(out)
    df.fold_softmax(again, o, l)
    assert torch.equal(again, out)
    return o, l, out, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 7, 8, 11, 16, 17, 40])
@pytest.mark.parametrize("rows,dim", [(1, 128), (33, 84), (257, 64), (5, 1), (3, 7), (100, 256), (2, 1000), (19, 130)])
def test_fold_softmax(env, dtype, W, rows, dim):
    _fold_case(env, W, (rows,), dim, dtype)
    _fold_case(env, W, (rows,), dim, dtype, empty=0.4, pad=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_fold_softmax_heads_and_far_lses(env, dtype):
    _fold_case(env, 4, (7, 6), 64, dtype, spread=60.0)
    _fold_case(env, 4, (3, 2, 5), 48, dtype, empty=0.9, pad=8)
    _fold_case(env, 4, (0,), 64, dtype)


def test_fold_softmax_large(env):
    _fold_case(env, 8, (30011,), 128, "f32", empty=0.2)


def test_fold_softmax_nan_and_infinite_lses(env):
    df, torch, dev = env
    outs = torch.randn((2, 4, 8), device=dev)
    lses = torch.tensor([[math.nan, math.inf, 1.0, -3e38], [0.0, 0.0, -1e4, -3e38]], device=dev)
    out, lse = torch.empty((4, 8), device=dev), torch.empty(4, device=dev)
    df.fold_softmax(out, outs, lses, lse=lse)
    assert torch.isnan(out).all(1).tolist() == [True, True, False, False]
    assert torch.isnan(lse).tolist() == [True, True, False, False]
    assert torch.equal(out[2], outs[0, 2]) and float(lse[2]) == 1.0
    assert torch.allclose(out[3], (outs[0, 3] + outs[1, 3]) / 2, rtol=0, atol=1e-6)


def test_two_ranks_join_to_the_whole(env):
    """A cache split over two ranks, attended apart and folded, against the whole."""
    df, torch, dev = env
    gen = _gen(torch, 5)
    k, v = (torch.randn((8, 16, 2, 64), generator=gen).to(dev) for _ in range(2))
    c = df.PagedCache(k, v)
    q = torch.randn((2, 4, 64), generator=gen).to(dev)
    table = torch.tensor([[1, 2, 3, 4], [5, 6, 7, 0]], dtype=torch.int32, device=dev)
    lens = torch.tensor([60, 33], dtype=torch.int32, device=dev)
    outs, lses = torch.empty((2, 2, 4, 64), device=dev), torch.empty((2, 2, 4), device=dev)
    df.attend_paged(outs[0], q, c, table[:, :2], lens.clamp(max=32), lse=lses[0])
    df.attend_paged(outs[1], q, c, table[:, 2:].contiguous(), (lens - 32).clamp(min=0), lse=lses[1])
    out, lse = torch.empty_like(q), torch.empty((2, 4), device=dev)
    df.fold_softmax(out, outs, lses, lse=lse)
    whole, wl = torch.empty_like(q), torch.empty((2, 4), device=dev)
    df.attend_paged(whole, q, c, table, lens, lse=wl)
    assert torch.allclose(out, whole, rtol=0, atol=3e-6) and torch.allclose(lse, wl, rtol=0, atol=3e-6)


# --------------------------------------------------------------------------
# refusals of the binding (the library's own are tested without a device)

def test_refusals(env):
    df, torch, dev = env
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    kc = torch.zeros((4, 16, 2, 64), device=dev, dtype=bf)
    vc = torch.zeros((4, 16, 2, 64), device=dev, dtype=bf)
    one = torch.ones(2, device=dev)
    for bad in (dict(k=kc.int()), dict(v=vc.float()), dict(v=vc[:3]), dict(k=kc.cpu(), v=vc.cpu()), dict(v=vc.cpu()),
                dict(k=kc.flatten(0, 1)), dict(k=kc.transpose(2, 3)), dict(k_scale=one),
                dict(k=kc.to(f8), v=vc.to(f8), k_scale=one.double()), dict(k=kc.to(f8), v=vc.to(f8), v_scale=one[:1])):
        with pytest.raises((TypeError, ValueError)):
            df.PagedCache(bad.get("k", kc), bad.get("v", vc), k_scale=bad.get("k_scale"), v_scale=bad.get("v_scale"))
    c = df.PagedCache(kc, vc)
    x, q = torch.zeros((3, 2, 64), device=dev, dtype=bf), torch.zeros((3, 4, 64), device=dev, dtype=bf)
    slots = torch.arange(3, device=dev)
    cs = torch.ones((9, 32), device=dev)
    good = dict(k=x, v=x, slots=slots)
    for bad in (dict(k=x.float()), dict(v=x[:2]), dict(k=x[:, :1]), dict(slots=slots.int()), dict(slots=slots[:2]),
                dict(slots=slots.cpu()), dict(q=q), dict(q_out=q), dict(q=q, q_out=q.float()), dict(q=q, q_out=q[:2]),
                dict(cos=cs), dict(cos=cs, sin=cs), dict(positions=slots), dict(cos=cs, sin=cs[:4], positions=slots),
                dict(cos=cs.double(), sin=cs, positions=slots), dict(k=x.cpu()), dict(k=x.transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            a = {**good, **bad}
            df.cache_append(c, a.pop("k"), a.pop("v"), a.pop("slots"), **a)
    with pytest.raises(df.DetfoldError) as e:  # more angles than the head has values
        df.cache_append(c, x, x, slots, cos=torch.ones((9, 33), device=dev), sin=torch.ones((9, 33), device=dev), positions=slots)
    assert e.value.rc == df.EINVAL
    with pytest.raises(df.DetfoldError) as e:  # the new keys lie in the cache itself
        df.cache_append(c, kc[0, :3], x, slots)
    assert e.value.rc == df.EOVERLAP
    table, lens = torch.zeros((3, 4), dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    good = dict(out=out, q=q, table=table, lens=lens)
    for bad in (dict(out=out.half()), dict(out=out[:2]), dict(q=q.half()), dict(q=q[0]), dict(table=table.long()),
                dict(table=table[:2]), dict(table=table.float()), dict(lens=lens.long()), dict(lens=lens.cpu()),
                dict(lse=torch.empty((3, 3), device=dev)), dict(lse=torch.empty((3, 4), device=dev).double()),
                dict(workspace=torch.empty(64)), dict(table=table.t()[:3]), dict(q=q[..., :32])):
        with pytest.raises((TypeError, ValueError, df.DetfoldError)):
            a = {**good, **bad}
            df.attend_paged(a.pop("out"), a.pop("q"), c, a.pop("table"), a.pop("lens"), **a)
    for bad in (dict(window=-1), dict(split=33), dict(split=-32), dict(max_len=-1), dict(scale=math.inf), dict(scale=math.nan)):
        with pytest.raises(df.DetfoldError) as e:
            df.attend_paged(out, q, c, table, lens, workspace=torch.empty(1 << 20, device=dev), **bad)
        assert e.value.rc == df.EINVAL
    with pytest.raises(df.DetfoldError) as e:
        df.attend_paged(q, q, c, table, lens)
    assert e.value.rc == df.EOVERLAP
    with pytest.raises(df.DetfoldError) as e:  # 3 query heads over 2
        df.attend_paged(out[:, :3], q[:, :3], c, table, lens)
    assert e.value.rc == df.EINVAL
    outs, lses = torch.zeros((2, 3, 8), device=dev), torch.zeros((2, 3), device=dev)
    o = torch.zeros((3, 8), device=dev)
    for bad in (dict(out=o.half()), dict(out=o[:2]), dict(out=o.cpu()), dict(lses=lses.half()), dict(lses=lses[:1]),
                dict(outs=outs.double()), dict(outs=outs.transpose(1, 2)), dict(outs=outs[:0], lses=lses[:0]),
                dict(lse=torch.zeros(2, device=dev)), dict(outs=outs.cpu())):
        with pytest.raises((TypeError, ValueError)):
            a = {**dict(out=o, outs=outs, lses=lses), **bad}
            df.fold_softmax(a.pop("out"), a.pop("outs"), a.pop("lses"), **a)
    with pytest.raises(df.DetfoldError) as e:
        df.fold_softmax(outs[0], outs, lses)
    assert e.value.rc == df.EOVERLAP
