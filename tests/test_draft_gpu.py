"""The drafted step's operators on the device (``attend_tree``, capped and biased
``attend_paged``, ``cache_copy``, ``cache_compact``) against their 64-bit forms
(``draft_oracle.py``, which derives the tolerances), at the sizes, layouts and masks
where they can go wrong, and a step of them together."""
import math
import random

import pytest

import decode_oracle
import draft_oracle as oracle
from test_decode_gpu import PAIRS, _cache, _gen, _normal, _scales, _t, _to, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _trees(rng, n, kind):
    """Masks and depths of one row's n drafted tokens."""
    if kind == "bits":  # any bits: not a tree, some see nothing, bits past the tree among them
        return [rng.choice([0, rng.getrandbits(64), rng.getrandbits(64) & rng.getrandbits(64), 1 << i]) for i in range(n)], \
            [rng.choice([rng.randint(0, 63), i, -5, 100]) for i in range(n)]
    masks, depths = [], []
    for i in range(n):
        parent = i - rng.randint(1, 4)
        masks.append((masks[parent] if parent >= 0 else 0) | 1 << i)
        depths.append(depths[parent] + 1 if parent >= 0 else 0)
    return masks, depths


def _signed(x):
    return x - 2 ** 64 if x >= 2 ** 63 else x


def _tree_case(env, lens, drafts, q_heads, heads, dim, v_dim, dtype, cache, page, order="thd", window=0, out=None,  # noqa: F811
               scale=None, split=0, spread=1.0, kind="tree", counts=None, cap=0.0, slopes=False, say=None, paged=False):
    """kind: "tree", "bits" or "chain" (no masks).  paged: drafts = 1 through attend_paged."""
    df, torch, dev = env
    seed = (lens, drafts, q_heads, heads, dim, v_dim, dtype, cache, page, order, window, out, kind, counts, cap, slopes)
    gen, rng = _gen(torch, *seed), random.Random(repr(seed))
    out_t = _t(torch, out or dtype)
    batch, top = len(lens), max(max(lens), 1)
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    host, _ = _cache(torch, gen, torch.device("cpu"), cache, pages, page, heads, dim, v_dim)
    ids = (torch.randperm(pages - 1, generator=gen) + 1).tolist()
    table = torch.full((batch, max(held) + 2), 2 ** 31 - 1, dtype=torch.int32)  # past a row's pages: never read
    trees = [_trees(rng, drafts, kind) for _ in lens]
    number = [drafts] * batch if counts is None else [min(max(n, 0), drafts) for n in counts]
    rows, mask = [], torch.zeros((pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        mine = [ids.pop() for _ in range(held[b])]
        table[b, :held[b]] = torch.tensor(mine, dtype=torch.int32)
        t = torch.arange(n)
        at = (torch.tensor(mine, dtype=torch.long)[t // page], t % page) if n else (t, t)
        depths = list(range(drafts)) if kind == "chain" else trees[b][1]
        seen, away = oracle.seen_by(drafts, n, number[b], None if kind == "chain" else trees[b][0], depths, window)
        seen = seen[:number[b]]
        rows.append((at, seen, away[:number[b]]))
        some = seen.any(0) if len(seen) else torch.zeros(n, dtype=torch.bool)
        mask[at[0][some], at[1][some]] = True
    for x in host:  # what no query sees is no number
        (x.view(torch.uint8) if cache == "e4m3" else x)[~mask] = 0x7F if cache == "e4m3" else math.nan
    views = [x.transpose(1, 2).contiguous().to(dev).transpose(1, 2) if order == "htd" else x.to(dev) for x in host]
    ks, vs = _scales(torch, gen, cache, heads, 1.0)
    wide = _normal(torch, gen, (batch, drafts, q_heads * dim + 8), dtype, spread)
    q = wide.to(dev)[..., :q_heads * dim].unflatten(2, (q_heads, dim))
    slope = (torch.rand(q_heads, generator=gen) - 0.1) * 0.2 if slopes else None
    c = df.PagedCache(*views, k_scale=_to(ks, dev), v_scale=_to(vs, dev))
    store = torch.full((batch, drafts, q_heads, v_dim + 8), 7.0, device=dev, dtype=out_t)
    o, lse = store[..., :v_dim], torch.full((batch, drafts, q_heads), 9.0, device=dev)
    ln, tab = torch.tensor(lens, dtype=torch.int32, device=dev), table.to(dev)
    args = dict(scale=scale, window=window, max_len=top, split=split, cap=cap, slopes=_to(slope, dev))
    if not paged:
        if counts is not None:
            args["counts"] = torch.tensor(counts, dtype=torch.int32, device=dev)
        if kind != "chain":
            args["masks"] = torch.tensor([[_signed(x) for x in m] for m, _ in trees], dtype=torch.int64, device=dev)
            if window or slopes:
                args["depths"] = torch.tensor([d for _, d in trees], dtype=torch.int32, device=dev)

    def call():
        if paged:
            df.attend_paged(o[:, 0], q[:, 0], c, tab, ln, lse=lse[:, 0], **args)
        else:
            df.attend_tree(o, q, c, tab, ln, lse=lse, **args)
    if say:
        print("case: tree %s" % (say,), flush=True)
    call()
    torch.cuda.synchronize()

    s, g = 1.0 / math.sqrt(dim) if scale is None else scale, q_heads // heads
    p_type = None if out_t == torch.float32 else out_t
    qd = wide[..., :q_heads * dim].unflatten(2, (q_heads, dim)).double()
    kd, vd = (x.double() * (1.0 if z is None else z.double()[:, None]) for x, z in zip(host, (ks, vs)))
    want = torch.full((batch, drafts, q_heads, v_dim), 7.0, dtype=torch.float64)
    wl = torch.full((batch, drafts, q_heads), 9.0, dtype=torch.float64)
    tol, tl = torch.zeros_like(want), torch.zeros_like(wl)
    for b, (at, seen, away) in enumerate(rows):
        for h in range(heads):
            i, n = slice(h * g, (h + 1) * g), number[b]
            want[b, :n, i], wl[b, :n, i], tol[b, :n, i], tl[b, :n, i] = oracle.attend(
                qd[b, :n, i], kd[at][:, h], vd[at][:, h], s, seen, away, cap, None if slope is None else slope[i].double(), out_t, p_type)
    decode_oracle.close(o, want, tol, "out")
    decode_oracle.close(lse, wl, tl, "lse")
    assert bool((store[..., v_dim:] == 7.0).all()), "written past the head"
    first = o.clone(), lse.clone()
    for _ in range(2):
        store.fill_(7.0), lse.fill_(9.0)
        call()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1]), "two calls differ"
    return c, q, tab, ln, o, lse, args


LENS = [0, 1, 5, 8, 9, 16, 31, 33, 64, 70, 129, 300]


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("out", [None, "f32"])
@pytest.mark.parametrize("order", ["thd", "htd"])
def test_tree_types(env, dtype, cache, out, order):  # noqa: F811
    _tree_case(env, LENS, 8, 8, 2, 128, 128, dtype, cache, 16, order, out=out)


@pytest.mark.parametrize("drafts", [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f32", "f32"), ("f16", "e4m3")])
@pytest.mark.parametrize("kind", ["tree", "bits", "chain"])
def test_tree_drafts(env, drafts, dtype, cache, kind):  # noqa: F811
    _tree_case(env, [0, 3, 64, 65, 130], drafts, 4, 2, 64, 64, dtype, cache, 16, kind=kind)
    _tree_case(env, [90, 64, 1, 0, 7], drafts, 6, 1, 128, 128, dtype, cache, 16, kind=kind, counts=[drafts, drafts // 2, 1, 2, 0])


@pytest.mark.parametrize("q_heads,heads,dim,v_dim,page,order,drafts", [
    (15, 3, 84, 84, 7, "thd", 5), (4, 4, 80, 64, 1, "htd", 9), (16, 1, 16, 16, 48, "thd", 3), (24, 1, 256, 128, 256, "htd", 4),
    (3, 3, 18, 22, 5, "htd", 33), (96, 2, 64, 256, 64, "thd", 2), (7, 1, 250, 246, 16, "thd", 6), (17, 1, 192, 64, 32, "htd", 11),
    (2, 2, 17, 19, 3, "thd", 64), (33, 1, 96, 96, 128, "thd", 2), (12, 12, 40, 132, 16, "thd", 8), (5, 1, 136, 72, 9, "htd", 20)])
@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_tree_shapes(env, q_heads, heads, dim, v_dim, page, order, drafts, dtype, cache):  # noqa: F811
    _tree_case(env, [0, 1, 30, 65, 200], drafts, q_heads, heads, dim, v_dim, dtype, cache, page, order)


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("window", [1, 3, 16, 33, 100, 400, 5000])
@pytest.mark.parametrize("kind", ["tree", "bits", "chain"])
def test_tree_window(env, dtype, cache, window, kind):  # noqa: F811
    _tree_case(env, [0, 1, 40, 64, 99, 100, 101, 417], 12, 6, 2, 64, 64, dtype, cache, 16, window=window, kind=kind)


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("cap,slopes", [(30.0, False), (0.0, True), (5.0, True), (1e-3, False), (1e30, False)])
def test_tree_scores(env, dtype, cache, cap, slopes):  # noqa: F811
    _tree_case(env, [0, 1, 50, 300], 10, 8, 2, 128, 128, dtype, cache, 16, cap=cap, slopes=slopes, spread=3.0)
    _tree_case(env, [40, 0, 50, 300], 6, 4, 1, 64, 64, dtype, cache, 16, cap=cap, slopes=slopes, spread=30.0, kind="bits", window=60)


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("cap,slopes", [(30.0, False), (0.0, True), (50.0, True)])
def test_paged_scores(env, dtype, cache, cap, slopes):  # noqa: F811
    """One new token a row, through attend_paged."""
    for out in (None, "f32"):
        _tree_case(env, LENS, 1, 8, 2, 128, 128, dtype, cache, 16, cap=cap, slopes=slopes, kind="chain", paged=True, out=out, spread=4.0)
    _tree_case(env, LENS, 1, 10, 2, 84, 80, dtype, cache, 7, cap=cap, slopes=slopes, kind="chain", paged=True, window=37)
    _tree_case(env, [3001, 12, 0], 1, 40, 2, 64, 64, dtype, cache, 16, cap=cap, slopes=slopes, kind="chain", paged=True, window=1500)


@pytest.mark.parametrize("dtype,cache,lens", [("bf16", "bf16", [5003]), ("f16", "e4m3", [20011, 3, 0, 7777]),
                                              ("f32", "f32", [4097, 1]), ("bf16", "e4m3", [30001])])
@pytest.mark.parametrize("split", [0, 32, 256, 4096])
@pytest.mark.parametrize("drafts", [3, 20])
def test_tree_long_and_split(env, dtype, cache, lens, split, drafts):  # noqa: F811
    _tree_case(env, lens, drafts, 8, 2, 128, 128, dtype, cache, 16, split=split)


@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_tree_sharp_and_flat(env, dtype, cache):  # noqa: F811
    _tree_case(env, [1, 50, 300], 8, 4, 1, 64, 64, dtype, cache, 16, spread=30.0)
    _tree_case(env, [1, 50, 300], 8, 4, 1, 64, 64, dtype, cache, 16, scale=0.0)
    _tree_case(env, [1, 50, 300], 8, 4, 1, 64, 64, dtype, cache, 16, scale=-0.3)


@pytest.mark.parametrize("seed", range(100))
def test_tree_random(env, seed):  # noqa: F811
    rng = random.Random(seed)
    log = lambda a, b: max(a, min(b, int(a * (b / a) ** rng.random())))  # noqa: E731
    heads = rng.choice([1, 1, 2, 3, 4, 5, 8])
    dim = rng.choice([64, 128, 256, rng.randint(16, 256), 16 * rng.randint(1, 16)])
    v_dim = rng.choice([dim, dim, rng.randint(16, 256)])
    q_heads = heads * rng.choice([1, 1, 2, 3, 4, 7, 8, 16, 17])
    (dtype, cache), page = rng.choice(PAIRS), rng.choice([1, 2, 5, 7, 16, 16, 32, 48, 64, 100])
    drafts, rows = rng.choice([1, 2, 3, 4, 8, 8, 16, 30, 64]), log(1, 20)
    longest = log(1, max(2, 600000 // (rows * heads * (dim + v_dim)))) + 40
    lens = [rng.choice([0, rng.randint(0, longest), longest, log(1, longest)]) for _ in range(rows)]
    counts = rng.choice([None, None, [rng.randint(-1, drafts + 1) for _ in lens]])
    cap, slopes = rng.choice([(0.0, False), (0.0, False), (20.0, False), (0.0, True), (50.0, True)])
    window, split = rng.choice([0, 0, 0, log(1, longest + 5)]), rng.choice([0, 0, 0, 32, 32 * rng.randint(1, 40)])
    out, kind = rng.choice([None, None, "f32"]), rng.choice(["tree", "tree", "bits", "chain"])
    case = (seed, lens, drafts, q_heads, heads, dim, v_dim, dtype, cache, page, window, split, out, kind, counts, cap, slopes)
    _tree_case(env, lens, drafts, q_heads, heads, dim, v_dim, dtype, cache, page, rng.choice(["thd", "htd"]), window=window, out=out,
               split=split, kind=kind, counts=counts, cap=cap, slopes=slopes, spread=rng.choice([1.0, 1.0, 4.0]), say=case)


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dim,group", [(64, 3), (84, 3), (256, 3), (128, 4), (80, 7), (128, 20)])
def test_tree_infinities_are_their_queries_alone(env, dtype, cache, what, dim, group):  # noqa: F811
    """A drafted value or key that is no number is in the results of those that see it, and in no other's; so is a
    prefix token's that a window hides from some."""
    df, torch, dev = env
    if cache == "e4m3" and not math.isnan(what):
        return  # 8 bits have no infinity
    gen = _gen(torch, dtype, cache, what, dim, group)
    t = _t(torch, cache)
    n, base, heads = 8, 40, 2
    k, v = (_normal(torch, gen, (4, 16, heads, dim), cache) for _ in range(2))
    masks = [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100001, 0b1000011, 0b10010101]
    depths = [0, 1, 1, 2, 2, 1, 2, 3]
    put = torch.tensor(what).to(t) if cache != "e4m3" else torch.tensor([0x7F], dtype=torch.uint8).view(t)[0]
    bits = (lambda x: x.view(torch.uint8)) if cache == "e4m3" else (lambda x: x)
    bits(v)[(base + 3) // 16, (base + 3) % 16, 0, 5] = bits(put.view(1))[0]   # drafted token 3, seen by 3 alone
    bits(v)[(base + 2) // 16, (base + 2) % 16, 1, 9] = bits(put.view(1))[0]   # 2: seen by 2, 4, 7
    bits(v)[1, 15, 0, 7] = bits(put.view(1))[0]                              # prefix token 31: within the window of depths 0 and 1
    bits(k)[(base + 5) // 16, (base + 5) % 16, 0, 3] = bits(put.view(1))[0]   # key of 5, seen by 5 alone
    q = _normal(torch, gen, (1, n, heads * group, dim), dtype)
    q[0, 5, :, 3] = q[0, 5, :, 3].abs() + 1
    c = df.PagedCache(k.to(dev), v.to(dev))
    table = torch.arange(4, dtype=torch.int32, device=dev)[None]
    lens = torch.tensor([base + n], dtype=torch.int32, device=dev)
    out, lse = torch.empty_like(q, device=dev), torch.empty((1, n, heads * group), device=dev)
    args = dict(masks=torch.tensor([masks], device=dev), depths=torch.tensor([depths], dtype=torch.int32, device=dev))
    df.attend_tree(out, q.to(dev), c, table, lens, lse=lse, window=11, **args)  # sees 11 positions: depth 1 from base - 9 on
    fine = torch.isfinite(out).cpu()[0]
    want = torch.ones_like(fine)
    want[3, :group, 5] = False
    for i in (2, 4, 7):
        want[i, group:, 9] = False
    for i in (0, 1, 2, 5):
        if depths[i] <= 1:
            want[i, :group, 7] = False
    if not (what == -math.inf):  # a key of -infinity takes no weight
        want[5, :group] = False
        assert not bool(torch.isfinite(lse)[0, 5, :group].any())
    assert torch.equal(fine, want), (torch.nonzero(fine != want)[:8],)
    ok = torch.ones((n, heads * group), dtype=torch.bool)
    if not (what == -math.inf):
        ok[5, :group] = False
    assert bool(torch.isfinite(lse).cpu()[0][ok].all())


@pytest.mark.parametrize("dtype,cache", PAIRS)
def test_tree_bad_rows_are_nan(env, dtype, cache):  # noqa: F811
    df, torch, dev = env
    gen = _gen(torch, 3)
    (_, _), views = _cache(torch, gen, dev, cache, 5, 16, 2, 64, 64)
    c = df.PagedCache(*views)
    n = 6
    q = _normal(torch, gen, (8, n, 4, 64), dtype).to(dev)
    good = [1, 2, 3, 4]
    table = torch.tensor([good, [1, 5, 3, 4], [1, 2, -1, 4], [1, 2, 3, 2 ** 31 - 1], good, good, good, good],
                         dtype=torch.int32, device=dev)
    lens = torch.tensor([64, 64, 64, 64, 65, 2 ** 31 - 1, -3, 50], dtype=torch.int32, device=dev)
    for split in (0, 32):
        out, lse = torch.empty_like(q), torch.empty((8, n, 4), device=dev)
        df.attend_tree(out, q, c, table, lens, max_len=100, lse=lse, split=split)
        bad = torch.isnan(out).cpu().flatten(1)
        assert bad.all(1).tolist() == [False, True, True, True, True, True, False, False]
        assert bad.any(1).tolist() == [False, True, True, True, True, True, False, False]
        assert bool((out[6] == 0).all()) and bool((lse[6] == -math.inf).all())
        assert torch.isnan(lse).cpu().flatten(1).all(1).tolist() == bad.all(1).tolist()
        df.attend_tree(out, q, c, table, lens, max_len=49, lse=lse, split=split)
        assert torch.isnan(out).cpu().flatten(1).all(1).tolist() == [True] * 6 + [False, True]


def test_tree_of_one_and_chains_agree_with_attend_paged(env):  # noqa: F811
    """A chain's token i sees what a single token of a row cut after it sees."""
    df, torch, dev = env
    c, q, table, lens, out, lse, _ = _tree_case(env, [200, 33, 77], 6, 8, 2, 128, 128, "f32", "f32", 16, kind="chain")
    for i in range(6):
        o, l = torch.empty_like(q[:, i]), torch.empty((3, 8), device=dev)
        df.attend_paged(o, q[:, i], c, table, lens - 5 + i, lse=l)
        assert torch.allclose(o, out[:, i], rtol=0, atol=4e-6) and torch.allclose(l, lse[:, i], rtol=0, atol=4e-6)


def test_tree_rows_alone_give_the_same_bits(env):  # noqa: F811
    df, torch, dev = env
    c, q, table, lens, out, lse, _ = _tree_case(env, [900, 33, 2000, 9], 9, 8, 2, 128, 128, "bf16", "bf16", 16, split=128, kind="chain")
    for b in range(4):
        o, l = torch.empty_like(q[:1]), torch.empty((1, 9, 8), device=dev)
        df.attend_tree(o, q[b:b + 1], c, table[b:b + 1], lens[b:b + 1], lse=l, split=128)
        assert torch.equal(o[0], out[b]) and torch.equal(l[0], lse[b])


def test_tree_far_pages_and_many_rows(env):  # noqa: F811
    """A cache of more than 2^32 bytes, and more rows than the device has workgroups for."""
    df, torch, dev = env
    pages = 280000
    kc = torch.zeros((pages, 16, 4, 128), device=dev, dtype=torch.bfloat16)
    c = df.PagedCache(kc, kc)
    k = torch.randn((3, 4, 128), device=dev).bfloat16()
    df.cache_append(c, k, k, torch.tensor([pages * 16 - 3, pages * 16 - 2, pages * 16 - 1], device=dev))
    q = torch.randn((1, 3, 8, 128), device=dev).bfloat16()
    out, table = torch.empty_like(q), torch.tensor([[pages - 1]], device=dev, dtype=torch.int32)
    masks = torch.tensor([[1, 2, 4]], device=dev)
    df.attend_tree(out, q, c, table, torch.tensor([16], device=dev, dtype=torch.int32), masks=masks, window=1,
                   depths=torch.tensor([[20, 20, 20]], dtype=torch.int32, device=dev))
    assert torch.equal(out[0], k.repeat_interleave(2, 1))  # each sees itself alone
    del kc, c
    torch.cuda.empty_cache()
    _tree_case(env, [20 + i % 30 for i in range(700)], 3, 2, 1, 64, 64, "bf16", "bf16", 16)


@pytest.mark.parametrize("drafts,q_heads,heads,dim,v_dim,page,order", [
    (13, 12, 2, 128, 128, 7, "thd"), (33, 4, 1, 80, 48, 16, "htd"), (64, 16, 2, 64, 64, 1, "thd"), (40, 8, 8, 112, 128, 33, "thd"),
    (64, 8, 1, 128, 64, 16, "htd"), (9, 32, 4, 32, 128, 64, "thd"), (20, 10, 1, 128, 16, 5, "thd"), (64, 3, 3, 96, 96, 16, "htd")])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("f16", "f16"), ("f16", "e4m3")])
def test_tree_many_queries(env, drafts, q_heads, heads, dim, v_dim, page, order, dtype, cache):  # noqa: F811
    """Key-value heads of many queries, whose tokens workgroups take from LDS."""
    _tree_case(env, [0, 1, drafts - 1, 64, 65, 90, 500], drafts, q_heads, heads, dim, v_dim, dtype, cache, page, order, kind="bits")
    _tree_case(env, [700, 3, 1200, 33], drafts, q_heads, heads, dim, v_dim, dtype, cache, page, order, window=100, cap=20.0, slopes=True,
               counts=[drafts, 2, drafts // 2, 0])
    _tree_case(env, [700, 1200], drafts, q_heads, heads, dim, v_dim, dtype, cache, page, order, split=96)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("drafts", [2, 8, 30])
def test_tree_lowest_scores(env, dtype, cache, drafts):  # noqa: F811
    """Keys of the type's lowest value and of -infinity: scores of -infinity take no weight beside others, and leave
    zeros where there is nothing else; with a cap they are -cap."""
    df, torch, dev = env
    t = _t(torch, cache)
    k = torch.zeros((4, 16, 1, 64), dtype=t)
    v = _normal(torch, _gen(torch, 31), (4, 16, 1, 64), cache)
    k[1, :, :, 0], k[2, :, :, 0] = -math.inf, torch.finfo(t).min
    q = torch.zeros((4, drafts, 4, 64), dtype=_t(torch, dtype))
    q[..., 0] = 1.0
    table = torch.tensor([[1, 1, 1], [2, 2, 2], [1, 3, 1], [2, 3, 2]], dtype=torch.int32, device=dev)
    lens = torch.tensor([40, 40, 40, 40], dtype=torch.int32, device=dev)
    c = df.PagedCache(k.to(dev), v.to(dev))
    masks = torch.ones((4, drafts), dtype=torch.int64, device=dev)  # the prefix and the first drafted token
    base = 40 - drafts
    keys, vals = k.double()[:, :, 0, 0], v.double()[:, :, 0]
    for cap in (0.0, 2.0):
        out, lse = torch.empty_like(q, device=dev), torch.empty((4, drafts, 4), device=dev)
        df.attend_tree(out, q.to(dev), c, table, lens, masks=masks, lse=lse, scale=2.0 ** -100, cap=cap)
        for b in range(4):
            pages = table[b].cpu().long()
            x = torch.cat([keys[p] for p in pages])[:base + 1] * 2.0 ** -100
            y = torch.cat([vals[p] for p in pages])[:base + 1]
            if cap:
                x = cap * torch.tanh(x / cap)
            p = torch.softmax(x, 0) if bool((x > -math.inf).any()) else torch.zeros_like(x)
            want = (p @ y).expand(drafts, 4, 64)
            tol = torch.full_like(want, 8 * torch.finfo(_t(torch, dtype)).eps * float(y.abs().max()))
            decode_oracle.close(out[b], want, tol, "out %d cap %g" % (b, cap))
            wl = torch.logsumexp(x, 0).expand(drafts, 4)
            decode_oracle.close(lse[b], wl, torch.where(torch.isfinite(wl), 1e-5 * (wl.abs() + 1), torch.zeros_like(wl)), "lse %d" % b)


def test_tree_two_streams_at_once(env):  # noqa: F811
    """Calls that overlap, each with a workspace of its own, and calls of many rows in parts of a fixed length."""
    df, torch, dev = env
    c, q, table, lens, out, lse, args = _tree_case(env, [3000, 500, 0, 2999], 8, 8, 2, 128, 128, "bf16", "bf16", 16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [(torch.empty_like(out), torch.empty_like(lse), df.attend_workspace(c, 4, 8, 3000, drafts=8)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (o, l, ws) in zip(streams, got):
            with torch.cuda.stream(s):
                df.attend_tree(o, q, c, table, lens, lse=l, workspace=ws, **args)
    torch.cuda.synchronize()
    for o, l, _ in got:
        assert torch.equal(o, out) and torch.equal(l, lse)
    with pytest.raises(df.DetfoldError) as e:
        df.attend_tree(got[0][0], q, c, table, lens, workspace=torch.empty(1024, dtype=torch.uint8, device=dev), **args)
    assert e.value.rc == df.ESIZE
    _tree_case(env, [10 + i * 7 % 900 for i in range(4200)], 2, 1, 1, 16, 16, "f32", "f32", 64)


def test_tree_nothing(env):  # noqa: F811
    df, torch, dev = env
    _tree_case(env, [0, 0], 4, 4, 2, 64, 64, "bf16", "bf16", 16)
    c = df.PagedCache(*(torch.zeros((1, 16, 2, 64), device=dev) for _ in range(2)))
    q = torch.zeros((0, 5, 4, 64), device=dev)
    i = torch.zeros((0,), dtype=torch.int32, device=dev)
    df.attend_tree(q.clone(), q, c, i.view(0, 1), i)
    q, i = torch.ones((2, 3, 4, 64), device=dev), torch.zeros((2,), dtype=torch.int32, device=dev)
    df.attend_tree(out := torch.ones_like(q), q, c, i.view(2, 1)[:, :0], i)  # a table of no pages
    assert bool((out == 0).all())


def test_tree_streams_and_graph(env):  # noqa: F811
    """On a stream of the caller's, and captured: every replay gives the eager bits."""
    df, torch, dev = env
    c, q, table, lens, out, lse, args = _tree_case(env, [3000, 0, 17, 2999], 8, 8, 2, 128, 128, "bf16", "bf16", 16, cap=30.0)
    want = out.clone(), lse.clone()
    ws = df.attend_workspace(c, 4, 8, 3000, drafts=8)
    o, l = torch.empty_like(want[0]), torch.empty_like(want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        df.attend_tree(o, q, c, table, lens, lse=l, workspace=ws, **args)
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    o.zero_()
    s.wait_stream(torch.cuda.current_stream())
    df.attend_tree(o, q, c, table, lens, lse=l, stream=s, **args)  # its own workspace, on a named stream
    s.synchronize()
    assert torch.equal(o, want[0])
    graph = torch.cuda.CUDAGraph()
    spare = torch.tensor([0, -1], dtype=torch.int32, device=dev)  # page 0 is no row's
    picks, counts = torch.zeros((4, 3), dtype=torch.int32, device=dev), torch.zeros(4, dtype=torch.int32, device=dev)
    with torch.cuda.graph(graph):
        df.cache_copy(c, lens[:1] * 0 + table[:1, 0], spare[:1])
        df.cache_compact(c, table, picks, counts)
        df.attend_tree(o, q, c, table, lens, lse=l, workspace=ws, **args)
    for _ in range(4):
        o.zero_(), l.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
        df.attend_tree(o, q, c, table, lens, lse=l, workspace=ws, **args)  # eager work between
        torch.cuda.synchronize()


# --------------------------------------------------------------------------
# cache_copy and cache_compact

def _bits(torch, x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


@pytest.mark.parametrize("heads,dim,v_dim,page,order,into", [
    (8, 128, 128, 16, "thd", None), (2, 64, 64, 16, "htd", None), (3, 84, 80, 7, "thd", "htd"), (1, 17, 19, 1, "thd", "thd"),
    (4, 16, 256, 64, "htd", "htd"), (5, 250, 18, 33, "pair", "thd"), (8, 128, 128, 16, "pair", None), (1, 33, 33, 5, "htd", "pair")])
@pytest.mark.parametrize("cache", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("part", [False, True])
def test_copy(env, heads, dim, v_dim, page, order, into, cache, part):  # noqa: F811
    df, torch, dev = env
    gen = _gen(torch, heads, dim, v_dim, page, order, into, cache, part)
    pages = 23
    host, views = _cache(torch, gen, dev, cache, pages, page, heads, dim, v_dim, order)
    c, w, target, on = df.PagedCache(*views), None, host, views
    if into:
        target, on = _cache(torch, gen, dev, cache, pages - 4, page, heads, dim, v_dim, into)
        w = df.PagedCache(*on)
    ids = torch.randperm(pages - 4, generator=gen).tolist()
    src, dst = ids[:7] + [-1, 3, 2 ** 31 - 1, pages], ids[7:14] + [ids[15], -1, ids[16], ids[17]]
    tokens = [(i * 5) % (page + 2) - 1 for i in range(len(src))] if part else None
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    df.cache_copy(c, i32(src), i32(dst), tokens=i32(tokens), into=w)
    torch.cuda.synchronize()
    for x, t, y in zip(host, target, on):
        want = oracle.copied(_bits(torch, x), _bits(torch, t), src, dst, tokens)
        assert torch.equal(_bits(torch, y.cpu().contiguous()), want)
    for x, y in zip(host, views):
        if into:
            assert torch.equal(_bits(torch, y.cpu().contiguous()), _bits(torch, x))


def test_copy_many_and_none(env):  # noqa: F811
    df, torch, dev = env
    gen = _gen(torch, 7)
    host, views = _cache(torch, gen, dev, "bf16", 9001, 4, 2, 64, 64)
    c = df.PagedCache(*views)
    ids = torch.randperm(9001, generator=gen).int()
    src, dst = ids[:4500].contiguous(), ids[4500:9000].contiguous()
    df.cache_copy(c, src.to(dev), dst.to(dev))
    for x, y in zip(host, views):
        x[dst.long()] = x[src.long()]
        assert torch.equal(y.cpu(), x)
    df.cache_copy(c, src[:0].to(dev), dst[:0].to(dev))
    for x, y in zip(host, views):
        assert torch.equal(y.cpu(), x)


def test_copy_far_pages(env):  # noqa: F811
    """Pages beyond 2^32 bytes."""
    df, torch, dev = env
    kc = torch.zeros((280000, 16, 4, 128), device=dev, dtype=torch.bfloat16)
    c = df.PagedCache(kc, kc)
    kc[3] = torch.randn((16, 4, 128), device=dev).bfloat16()
    df.cache_copy(c, torch.tensor([3], dtype=torch.int32, device=dev), torch.tensor([279999], dtype=torch.int32, device=dev))
    assert torch.equal(kc[279999], kc[3]) and not bool(kc[279998].any())
    table = torch.tensor([[279999, 7]], dtype=torch.int32, device=dev)
    df.cache_compact(c, table, torch.tensor([[5, 15]], dtype=torch.int32, device=dev), torch.tensor([2], dtype=torch.int32, device=dev))
    assert torch.equal(kc[279999, :2], kc[3, [5, 15]]) and torch.equal(kc[279999, 2:], kc[3, 2:])
    del kc, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("heads,dim,v_dim,page,order", [
    (8, 128, 128, 16, "thd"), (2, 64, 64, 16, "htd"), (3, 84, 80, 7, "thd"), (1, 17, 19, 1, "thd"), (4, 16, 256, 64, "htd"),
    (5, 250, 18, 33, "pair"), (2, 256, 256, 16, "thd")])
@pytest.mark.parametrize("cache", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("apart", [False, True])
def test_compact(env, heads, dim, v_dim, page, order, cache, apart):  # noqa: F811
    df, torch, dev = env
    gen, rng = _gen(torch, heads, dim, v_dim, page, order, cache, apart), random.Random(heads * dim + page + apart)
    lens = [400, 1, 64, 65, 130, 200, 17]
    held = [-(-n // page) for n in lens]
    pages = sum(held) * (2 if apart else 1) + 5
    host, views = _cache(torch, gen, dev, cache, pages, page, heads, dim, v_dim, order)
    ids = torch.randperm(pages - 1, generator=gen).add(1).tolist()
    wide = max(held)
    table, to = ([[ids.pop() for _ in range(n)] + [0] * (wide - n) for n in held] if side else None for side in (True, apart))
    starts = [0, 0, 5, 40, 3, 150, -2]
    most = 330
    picks = [sorted(rng.sample(range(n - max(s, 0)), min(n - max(s, 0), rng.randint(1, n)))) for n, s in zip(lens, starts)]
    counts = [len(p) for p in picks]
    picks[0] = [rng.randrange(400) for _ in range(300)]     # in no order, some twice, some below their own place
    counts[0], counts[4] = 300, most + 7                    # more than there are: as many as there are
    picks[4] = [x if x < 120 else rng.choice([-1, 10 ** 9, 2 ** 31 - 1]) for x in range(most)]
    counts[1] = -3
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    padded = [p + [0] * (most - len(p)) for p in picks]
    c = df.PagedCache(*views)
    args = dict(starts=i32(starts))
    if apart:
        args["to"] = i32(to)
    df.cache_compact(c, i32(table), i32(padded), i32(counts), **args)
    torch.cuda.synchronize()
    for x, y in zip(host, views):
        want = oracle.compacted(_bits(torch, x), table, padded, counts, starts, to)
        assert torch.equal(_bits(torch, y.cpu().contiguous()), want)


def test_compact_long_in_place(env):  # noqa: F811
    """Many tiles of moves, whose sources and targets interleave; and pages outside the cache."""
    df, torch, dev = env
    gen, rng = _gen(torch, 11), random.Random(11)
    host, views = _cache(torch, gen, dev, "bf16", 520, 16, 2, 64, 64)
    c = df.PagedCache(*views)
    table = [list(range(256)), list(range(256, 512))]
    table[1][3], table[1][200] = 520, -1
    picks = [list(range(1, 4001)), sorted(rng.sample(range(4096), 3000)) + [0] * 1000]
    counts = [4000, 3000]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    df.cache_compact(c, i32(table), i32(picks), i32(counts))
    torch.cuda.synchronize()
    for x, y in zip(host, views):
        assert torch.equal(y.cpu(), oracle.compacted(x, table, picks, counts, None, None))


# --------------------------------------------------------------------------
# the step as it is used

@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_drafted_step(env, cache):  # noqa: F811
    """Trees are appended, attended and cut down to an accepted path, step after step, with a fork of one request on
    the way: the caches hold what one token after another would have left, bit for bit, and the accepted tokens'
    attention is that of single tokens."""
    df, torch, dev = env
    gen, rng = _gen(torch, cache, 21), random.Random(21)
    batch, n, hq, h, d, page, wide = 3, 9, 4, 2, 64, 16, 12
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731

    def fresh():
        k, v = (torch.zeros((1 + 4 * wide, page, h, d), device=dev).to(_t(torch, cache)) for _ in range(2))
        return df.PagedCache(k, v)
    ours, plain = fresh(), fresh()
    table = (torch.arange(4 * wide, device=dev, dtype=torch.int32) + 1).view(4, wide)
    angle = torch.arange(200, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))
    turn = dict(cos=angle.cos().float().to(dev), sin=angle.sin().float().to(dev))
    length = [0, 0, 0]
    slot = lambda b, t: int(table[b, t // page]) * page + t % page  # noqa: E731
    for step in range(8):
        if step == 5:  # row 1 forks into pages of row 3, which takes its place: whole pages and a part of the last
            held = -(-length[1] // page)
            tokens = [min(page, length[1] - page * i) for i in range(held)]
            for c in (ours, plain):
                df.cache_copy(c, table[1, :held].contiguous(), table[3, :held].contiguous(), tokens=i32(tokens))
            table[1] = table[3]
        trees = [_trees(rng, n, "tree") for _ in range(batch)]
        count = [rng.randint(1, n) for _ in range(batch)]
        q, k, v = (torch.randn((batch * n, x, d), generator=gen).bfloat16().to(dev) for x in (hq, h, h))
        real = [i < count[b] for b in range(batch) for i in range(n)]
        slots = [slot(b, length[b] + i) if i < count[b] else -1 for b in range(batch) for i in range(n)]
        at = torch.tensor([length[b] + trees[b][1][i] for b in range(batch) for i in range(n)], device=dev)
        turned = torch.empty_like(q)
        df.cache_append(ours, k, v, torch.tensor(slots, device=dev), q=q, q_out=turned, positions=at, **turn)
        lens = i32([length[b] + count[b] for b in range(batch)])
        out, lse = (torch.full(s, 7.0, device=dev) for s in ((batch, n, hq, d), (batch, n, hq)))
        df.attend_tree(out, turned.view(batch, n, hq, d), ours, table[:batch], lens, counts=i32(count), lse=lse,
                       masks=torch.tensor([[_signed(x) for x in m] for m, _ in trees], device=dev),
                       depths=i32([t for _, t in trees]))
        assert bool((out.view(-1, hq, d)[~torch.tensor(real)] == 7.0).all())
        # each row keeps one branch: the path to a drafted token
        paths = []
        for b in range(batch):
            leaf = rng.randrange(count[b])
            paths.append([j for j in range(n) if trees[b][0][leaf] >> j & 1])
        df.cache_compact(ours, table[:batch].contiguous(), i32([p + [0] * (n - len(p)) for p in paths]), i32([len(p) for p in paths]),
                         starts=i32(length))
        # the same path, token after token
        for j in range(n):
            rows = [b for b in range(batch) if j < len(paths[b])]
            if not rows:
                break
            take = torch.tensor([b * n + paths[b][j] for b in rows], device=dev)
            turned1 = torch.empty_like(q[take])
            df.cache_append(plain, k[take], v[take], torch.tensor([slot(b, length[b] + j) for b in rows], device=dev), q=q[take],
                            q_out=turned1, positions=torch.tensor([length[b] + j for b in rows], device=dev), **turn)
            one, l1 = torch.empty((len(rows), hq, d), device=dev), torch.empty((len(rows), hq), device=dev)
            df.attend_paged(one, turned1, plain, table[rows].contiguous(), i32([length[b] + j + 1 for b in rows]), lse=l1)
            for r, b in enumerate(rows):
                assert torch.allclose(one[r], out[b, paths[b][j]], rtol=0, atol=1e-5)
                assert torch.allclose(l1[r], lse[b, paths[b][j]], rtol=0, atol=1e-5)
        length = [length[b] + len(paths[b]) for b in range(batch)]
        for b in range(batch):
            own = torch.tensor([slot(b, t) for t in range(length[b])], device=dev)
            for x, y in ((ours.k, plain.k), (ours.v, plain.v)):
                assert torch.equal(_bits(torch, x).flatten(0, 1)[own], _bits(torch, y).flatten(0, 1)[own]), (step, b)


# --------------------------------------------------------------------------
# refusals of the binding (the library's own are tested without a device)

def test_refusals(env):  # noqa: F811
    df, torch, dev = env
    bf = torch.bfloat16
    c = df.PagedCache(*(torch.zeros((4, 16, 2, 64), device=dev, dtype=bf) for _ in range(2)))
    q = torch.zeros((3, 5, 4, 64), device=dev, dtype=bf)
    out, lse = torch.empty_like(q), torch.empty((3, 5, 4), device=dev)
    table, lens = torch.zeros((3, 4), dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    masks, depths = torch.zeros((3, 5), dtype=torch.int64, device=dev), torch.zeros((3, 5), dtype=torch.int32, device=dev)
    slopes = torch.zeros(4, device=dev)
    good = dict(out=out, q=q, table=table, lens=lens)
    for bad in (dict(out=out.half()), dict(out=out[:2]), dict(out=out[:, :4]), dict(q=q.half()), dict(q=q[0]), dict(q=q[:, :0], out=out[:, :0]),
                dict(table=table.long()), dict(table=table[:2]), dict(lens=lens.long()), dict(lens=lens.cpu()), dict(lse=lse[:, :4]),
                dict(lse=lse.double()), dict(masks=masks.int()), dict(masks=masks[:, :4]), dict(masks=masks.cpu()),
                dict(counts=lens.long()), dict(counts=lens[:2]), dict(depths=depths.long()), dict(depths=depths[:, :3]),
                dict(slopes=slopes.half()), dict(slopes=slopes[:3]), dict(masks=masks, window=4), dict(masks=masks, slopes=slopes),
                dict(workspace=torch.empty(64)), dict(q=q[..., :32]), dict(q=q.transpose(2, 3)),
                dict(q=torch.zeros((3, 65, 4, 64), device=dev, dtype=bf), out=torch.zeros((3, 65, 4, 64), device=dev, dtype=bf))):
        with pytest.raises((TypeError, ValueError)):
            a = {**good, **bad}
            df.attend_tree(a.pop("out"), a.pop("q"), c, a.pop("table"), a.pop("lens"), **a)
    for bad in (dict(window=-1), dict(split=33), dict(max_len=-1), dict(scale=math.inf), dict(cap=-1.0), dict(cap=math.inf),
                dict(cap=math.nan), dict(cap=1e300)):
        with pytest.raises((df.DetfoldError, OverflowError)) as e:
            df.attend_tree(out, q, c, table, lens, workspace=torch.empty(1 << 22, device=dev), **bad)
        assert getattr(e.value, "rc", df.EINVAL) == df.EINVAL
    with pytest.raises(df.DetfoldError) as e:
        df.attend_tree(q, q, c, table, lens)
    assert e.value.rc == df.EOVERLAP
    one, o1 = q[:, 0].contiguous(), out[:, 0].contiguous()
    for bad in (dict(q=q), dict(out=out), dict(lse=lse), dict(slopes=slopes[:3]), dict(slopes=slopes.double())):
        with pytest.raises((TypeError, ValueError)):
            a = {**dict(out=o1, q=one, slopes=slopes), **bad}
            df.attend_paged(a.pop("out"), a.pop("q"), c, table, lens, **a)
    for bad in (dict(cap=-2.0), dict(cap=math.nan)):
        with pytest.raises(df.DetfoldError) as e:
            df.attend_paged(o1, one, c, table, lens, **bad)
        assert e.value.rc == df.EINVAL
    i = torch.zeros(2, dtype=torch.int32, device=dev)
    other = df.PagedCache(*(torch.zeros((4, 8, 2, 64), device=dev, dtype=bf) for _ in range(2)))
    for bad in (dict(src=i.long()), dict(src=i[:1]), dict(dst=None), dict(dst=i.cpu()), dict(tokens=i.long()), dict(tokens=i[:1]),
                dict(src=i.view(1, 2)), dict(into=other)):
        with pytest.raises((TypeError, ValueError)):
            a = {**dict(src=i, dst=i), **bad}
            df.cache_copy(c, a.pop("src"), a.pop("dst"), **a)
    shared = df.PagedCache(c.k[:2], torch.zeros((2, 16, 2, 64), device=dev, dtype=bf))
    with pytest.raises(df.DetfoldError) as e:
        df.cache_copy(c, i, i, into=shared)
    assert e.value.rc == df.EOVERLAP
    picks = torch.zeros((3, 2), dtype=torch.int32, device=dev)
    for bad in (dict(picks=picks.long()), dict(picks=picks[0]), dict(picks=picks[:2]), dict(counts=lens[:2]), dict(counts=lens.cpu()),
                dict(starts=lens.long()), dict(table=table.long()), dict(table=table[:2]), dict(to=table.long()), dict(to=table[:2])):
        with pytest.raises((TypeError, ValueError)):
            a = {**dict(table=table, picks=picks, counts=lens), **bad}
            df.cache_compact(c, a.pop("table"), a.pop("picks"), a.pop("counts"), **a)
