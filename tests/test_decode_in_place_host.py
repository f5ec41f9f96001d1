"""Queries turned in place (q_out is q) beside keys and values of the same buffer
(CPU only, launches recorded): accepted where no element is shared, refused where
one is, since its query's store and its key's load would race."""
import random

import pytest

from decode_recorder import recorder  # noqa: F401
from test_decode_host import append, cache

OK, EOVERLAP = 0, 2
BASE = 0x7FA000000000  # away from what the other buffers have


def _call(lib, q, k, v, tokens, heads, dim, v_dim):
    """q, k, v: (offset, token, head, heads) in elements of a bfloat16 buffer."""
    c = cache(heads=heads, dim=dim, v_dim=v_dim, k_head=dim, k_token=dim * heads, k_page=16 * dim * heads, v_head=v_dim,
              v_token=v_dim * heads, v_page=16 * v_dim * heads)
    at = [BASE + 2 * x[0] for x in (q, k, v)]
    return lib.detfold_cache_append(c, append(q=at[0], q_out=at[0], k=at[1], v=at[2], tokens=tokens, q_token=q[1], out_token=q[1],
                                              q_head=q[2], out_head=q[2], q_heads=q[3], k_token=k[1], k_head=k[2],
                                              v_token=v[1], v_head=v[2], rot=16), None)


def _elements(x, tokens, dim):
    return {x[0] + t * x[1] + h * x[2] + i for t in range(tokens) for h in range(x[3]) for i in range(dim)}


def test_views_of_one_projection(recorder):  # noqa: F811
    for tokens in (1, 2, 67, 8192, 1 << 20):
        for hq, h, d, dv in ((8, 2, 64, 64), (32, 8, 128, 128), (15, 3, 84, 80), (1, 1, 16, 16)):
            width = hq * d + h * (d + dv)
            order = [("q", hq, d), ("k", h, d), ("v", h, dv)]
            for turn in range(3):
                at, off = {}, 0
                for name, n, dim in order[turn:] + order[:turn]:
                    at[name] = (off, width, dim, n)
                    off += n * dim
                assert _call(recorder, at["q"], at["k"], at["v"], tokens, h, d, dv) == OK


def test_head_by_head(recorder):  # noqa: F811
    """[tokens, heads, query | key | value]: the heads interleave too."""
    for tokens in (1, 5, 4096):
        for h, d in ((4, 64), (8, 128)):
            views = [(i * d, 3 * h * d, 3 * d, h) for i in range(3)]
            assert _call(recorder, *views, tokens, h, d, d) == OK


def test_head_major(recorder):  # noqa: F811
    """[heads, tokens, dim]: a token is nearer than a head."""
    n, d = 33, 64
    assert _call(recorder, (0, d, n * d, 4), (4 * n * d, d, n * d, 2), (6 * n * d, d, n * d, 2), n, 2, d, d) == OK


@pytest.mark.parametrize("tokens", [1, 2, 67])
@pytest.mark.parametrize("which", ["k", "v"])
def test_shared_elements(recorder, tokens, which):  # noqa: F811
    hq, h, d = 8, 2, 64
    width = hq * d + 2 * h * d
    q, k, v = (0, width, d, hq), (hq * d, width, d, h), ((hq + h) * d, width, d, h)
    for bad in (0, d, (hq - h) * d, (hq - h + 1) * d, (hq - h) * d + 1, hq * d - 1, 1):
        views = dict(k=k, v=v)
        views[which] = (bad, width, d, h)
        assert _call(recorder, q, views["k"], views["v"], tokens, h, d, d) == EOVERLAP, bad
    if tokens > 1:  # a key's second token in the query's
        views = dict(k=k, v=v)
        views[which] = (hq * d, width - 1, d, h)
        assert _call(recorder, q, views["k"], views["v"], tokens, h, d, d) == EOVERLAP
        # the last heads of a key reach the next token's queries
        views[which] = (width - d - 5, width, d, h)
        assert _call(recorder, q, views["k"], views["v"], tokens, h, d, d) == EOVERLAP


def test_against_the_sets_of_elements(recorder):  # noqa: F811
    """Random layouts: accepted exactly where the sets are disjoint, if the tokens
    are equally far apart."""
    rng = random.Random(61)
    seen = {OK: 0, EOVERLAP: 0}
    while min(seen.values()) < 400:
        tokens, hq, h, d, dv = rng.randint(1, 6), rng.randint(1, 4), rng.randint(1, 3), rng.choice([16, 17, 20]), rng.choice([16, 18])
        hq = h * rng.randint(1, 2)
        token = rng.randint(16, 400)
        gap = lambda n: rng.choice([n, n + rng.randint(0, 40), 2 * n, token * tokens, rng.randint(0, 60)])  # noqa: E731
        q, k, v = ((rng.randint(0, 300), token, gap(dim), n) for dim, n in ((d, hq), (d, h), (dv, h)))
        mine = _elements(q, tokens, d)
        if len(mine) < tokens * hq * d:
            continue  # q_out itself meets itself: refused as such
        got = _call(recorder, q, k, v, tokens, h, d, dv)
        shared = bool(mine & (_elements(k, tokens, d) | _elements(v, tokens, dv)))
        if not shared and got == EOVERLAP and not _nested(q, tokens, d):
            continue  # a layout of q_out that is not told from one that meets itself
        assert got == (EOVERLAP if shared else OK), (q, k, v, tokens, hq, h, d, dv)
        seen[got] += 1


def _nested(x, tokens, dim):
    """Heads within a token, or tokens within a head."""
    (_, t, s, n) = x
    if tokens > 1 and n > 1:
        return (s >= dim and t >= (n - 1) * s + dim) or (t >= dim and s >= (tokens - 1) * t + dim)
    return True
