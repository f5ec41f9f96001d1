"""The compaction in place on caches whose keys and values, or heads, lie in each other's
memory (CPU only, launches recorded).  Each run of a token moves in a workgroup of its
own and nothing orders them: accepted where no two of them share an element, with what
is the same memory moved once, and refused else."""
import random

import pytest

from draft_recorder import draft_recorder  # noqa: F401
from test_decode_host import BF, E4, F32, cache
from test_draft_host import compact

OK, EOVERLAP = 0, 2
BASE = 0x7FA000000000  # away from what the lists have


def _call(lib, k, v, pages, page, heads, dim, v_dim, type=BF):
    """k, v: (offset, page, token, head) in elements.  The result, and the runs that move: of keys and of values."""
    size = {BF: 2, E4: 1, F32: 4}[type]
    c = cache(k=BASE + size * k[0], v=BASE + size * v[0], pages=pages, page=page, heads=heads, dim=dim, v_dim=v_dim, k_page=k[1],
              k_token=k[2], k_head=k[3], v_page=v[1], v_token=v[2], v_head=v[3], type=type)
    before = lib.recorded_moves()
    rc = lib.detfold_cache_compact(c, compact(to=0), None)
    assert lib.recorded_moves() == before + (rc == OK)
    keys = lib.recorded_key_runs()
    return rc, (keys, lib.recorded_runs() - keys) if rc == OK else None


def _thd(at, page, heads, dim, wide=0):
    return at, page * (wide or heads * dim), wide or heads * dim, dim


@pytest.mark.parametrize("type", [BF, E4, F32])
def test_pools_of_their_own(draft_recorder, type):  # noqa: F811
    for pages, page, heads, dim, v_dim in ((9, 16, 8, 128, 128), (1, 1, 1, 16, 16), (5, 7, 3, 84, 80), (700000, 16, 4, 128, 64), (3, 64, 4, 16, 256)):
        args = pages, page, heads, dim, v_dim, type
        both = OK, (heads, heads)
        k, far = _thd(0, page, heads, dim), pages * page * heads * dim
        assert _call(draft_recorder, k, _thd(far, page, heads, v_dim), *args) == both
        htd = 0, page * heads * dim, dim, page * dim
        assert _call(draft_recorder, htd, (far, page * heads * v_dim, v_dim, page * v_dim), *args) == both
        assert _call(draft_recorder, htd, _thd(far, page, heads, v_dim), *args) == both
        # one tensor: keys and values side by side in a head, a token, a page, and behind each other
        w = dim + v_dim
        assert _call(draft_recorder, (0, page * heads * w, heads * w, w), (dim, page * heads * w, heads * w, w), *args) == both
        assert _call(draft_recorder, (0, page * heads * w, heads * w, dim), (heads * dim, page * heads * w, heads * w, v_dim), *args) == both
        assert _call(draft_recorder, (0, page * heads * w, heads * dim, dim), (page * heads * dim, page * heads * w, heads * v_dim, v_dim), *args) == both
        assert _call(draft_recorder, (heads * v_dim, page * heads * w, heads * w, dim), (0, page * heads * w, heads * w, v_dim), *args) == both
        # a layer's share of a tensor of several
        assert _call(draft_recorder, (0, 4 * page * heads * w, heads * w, w), (dim, 4 * page * heads * w, heads * w, w), *args) == both


@pytest.mark.parametrize("type", [BF, E4, F32])
def test_one_memory_moves_once(draft_recorder, type):  # noqa: F811
    for pages, page, heads, dim in ((9, 16, 8, 128), (1, 1, 1, 16), (5, 7, 3, 84), (700000, 16, 4, 128)):
        k = _thd(0, page, heads, dim)
        assert _call(draft_recorder, k, k, pages, page, heads, dim, dim, type) == (OK, (heads, 0))
        assert _call(draft_recorder, k, k, pages, page, heads, dim, 16, type) == (OK, (heads, 0))
        assert _call(draft_recorder, (0, page * dim * heads, dim, page * dim), (dim - 16, page * dim * heads, dim, page * dim), pages, page,
                     heads, dim, 16, type) == (OK, (heads, 0))
        if dim > 16:
            assert _call(draft_recorder, (3, *k[1:]), k, pages, page, heads, 16, dim, type) == (OK, (0, heads))
        # heads that are one
        one = 0, page * dim, dim, 0
        far = pages * page * dim, page * dim, dim, 0
        assert _call(draft_recorder, one, far, pages, page, heads, dim, dim, type) == (OK, (1, 1))
        assert _call(draft_recorder, one, one, pages, page, heads, dim, dim, type) == (OK, (1, 0))
        assert _call(draft_recorder, one, _thd(pages * page * dim, page, heads, dim), pages, page, heads, dim, dim, type) == (OK, (1, heads))


def test_other_sharing_is_refused(draft_recorder):  # noqa: F811
    pages, page, heads, dim = 9, 16, 4, 64
    k = _thd(0, page, heads, dim)
    token, whole = heads * dim, page * heads * dim
    for at in (1, dim - 1, dim, token, token + dim, whole, 8 * whole, 9 * whole - 1):  # a part, another head, token or page
        assert _call(draft_recorder, k, (at, *k[1:]), pages, page, heads, dim, dim) == (EOVERLAP, None), at
        assert _call(draft_recorder, (at, *k[1:]), k, pages, page, heads, dim, dim) == (EOVERLAP, None), at
    far = _thd(10 * whole, page, heads, dim)
    for bad in ((0, whole, token, dim - 1), (0, whole, 0, dim), (0, 0, token, dim), (0, whole - 1, token, dim), (0, whole, token - 1, dim),
                (0, whole, dim, dim), (0, dim, token, dim)):
        assert _call(draft_recorder, bad, far, pages, page, heads, dim, dim) == (EOVERLAP, None), bad
        assert _call(draft_recorder, far, bad, pages, page, heads, dim, dim) == (EOVERLAP, None), bad
    # expanded keys beside values of their own in the same memory; other orders of the same memory
    assert _call(draft_recorder, (0, whole, token, 0), k, pages, page, heads, dim, dim) == (EOVERLAP, None)
    assert _call(draft_recorder, k, (0, whole, dim, page * dim), pages, page, heads, dim, dim) == (EOVERLAP, None)
    # values behind the last key of a narrower pool reach back by their heads
    assert _call(draft_recorder, (5 * 10 ** 6, whole, token, dim), (0, whole, token, 25 * 10 ** 5), pages, page, 3, dim, dim) == (EOVERLAP, None)


def test_into_other_pages_any_pool_will_do(draft_recorder):  # noqa: F811
    lib, before = draft_recorder, draft_recorder.recorded_moves()
    k = BASE
    assert lib.detfold_cache_compact(cache(k=k, v=k, v_dim=64, v_page=2048, v_token=128, v_head=64), compact(), None) == OK
    assert lib.recorded_moves() == before + 1


def _runs(x, pages, page, heads, dim):
    return {(p, t, h): range(x[0] + p * x[1] + t * x[2] + h * x[3], x[0] + p * x[1] + t * x[2] + h * x[3] + dim)
            for p in range(pages) for t in range(page) for h in range(heads)}


def test_against_the_sets_of_elements(draft_recorder):  # noqa: F811
    """Random layouts: what is accepted is safe, and what is not is not, or not told from it."""
    rng = random.Random(83)
    seen = {(OK, True): 0, (OK, False): 0, (EOVERLAP, True): 0, (EOVERLAP, False): 0}
    tried = 0
    while tried < 6000 or min(seen[OK, True], seen[OK, False], seen[EOVERLAP, False]) < 60:
        tried += 1
        pages, page, heads, dim, v_dim = rng.randint(1, 3), rng.randint(1, 3), rng.randint(1, 3), rng.choice([16, 17, 20]), rng.choice([16, 17, 24])

        def layout(d):
            order, s, at = [0, 1, 2], {}, d + rng.choice([0, 0, rng.randint(0, 30)])
            rng.shuffle(order)
            n = (pages, page, heads)
            for i in order:
                s[i] = at
                at = at * n[i] + rng.choice([0, 0, rng.randint(0, 30)])
            if rng.random() < 0.15:
                s[rng.randrange(3)] = rng.choice([0, 0, rng.randint(0, 60)])
            return [s[0], s[1], s[2]]
        ks = layout(max(dim, v_dim) if rng.random() < 0.5 else dim + v_dim)
        vs = ks if rng.random() < 0.7 else layout(v_dim)
        k, v = (300, *ks), (300 + rng.choice([0, 0, dim, rng.randint(-30, 30), rng.randint(-200, 400), *ks, 900]), *vs)
        rc, moved = _call(draft_recorder, k, v, pages, page, heads, dim, v_dim)
        one_k, one_v = ks[2] == 0, vs[2] == 0
        kr, vr = _runs(k, pages, page, 1 if one_k else heads, dim), _runs(v, pages, page, 1 if one_v else heads, v_dim)

        def distinct(*sets):
            every = [e for s in sets for r in s.values() for e in r]
            return len(every) == len(set(every))
        apart = distinct(kr, vr)
        inside = (kr.keys() == vr.keys() and distinct(kr) and all(set(vr[i]) <= set(kr[i]) for i in kr))
        around = (kr.keys() == vr.keys() and distinct(vr) and all(set(kr[i]) <= set(vr[i]) for i in kr))
        want = (len(kr) // pages // page if not around or inside else 0, len(vr) // pages // page if not inside else 0)
        if rc == OK:
            assert apart or inside or around, (k, v, pages, page, heads, dim, v_dim)
            assert moved == want, (k, v, moved, want)
        elif apart or inside or around:
            # of other strides in one span, or in an order that is not told from sharing
            n = (pages, page, heads)
            alike = all(a == b or m == 1 for a, b, m in zip(ks, vs, n)) and one_k == one_v

            def nested(s, d):
                at = d
                for x, m in sorted((x, m) for x, m in zip(s, n) if m > 1 and x):
                    if x < at:
                        return False
                    at += x * (m - 1)
                return True
            assert not alike or not nested(ks, dim) or not nested(vs, v_dim), (k, v, pages, page, heads, dim, v_dim)
        seen[rc, apart] += 1
    assert seen[EOVERLAP, True] < tried // 5, seen
