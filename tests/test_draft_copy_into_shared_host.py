"""Copies into another pool whose keys and values, or heads, are one memory (CPU only,
launches recorded): accepted from pools where they are so too, refused from others,
whose two values would go to the same place in no order."""
import pytest

from draft_recorder import draft_recorder  # noqa: F401
from test_decode_host import BF, E4, F32, cache
from test_draft_host import SIDE

OK, EOVERLAP = 0, 2
ONE, OTHER = 0x7FA000000000, 0x7FB000000000
PAGE, HEADS, DIM = 16, 4, 64
TOKEN = HEADS * DIM
WHOLE = PAGE * TOKEN


def _pool(base, k, v, type, v_dim):
    """k, v: (offset, page, token, head) in elements."""
    size = {BF: 2, E4: 1, F32: 4}[type]
    return cache(k=base + size * k[0], v=base + size * v[0], pages=9, page=PAGE, heads=HEADS, dim=DIM, v_dim=v_dim, k_page=k[1],
                 k_token=k[2], k_head=k[3], v_page=v[1], v_token=v[2], v_head=v[3], type=type)


def _kinds(v_dim):
    thd = (WHOLE, TOKEN, DIM)
    return {
        "apart": ((0, *thd), (9 * WHOLE, PAGE * HEADS * v_dim, HEADS * v_dim, v_dim)),
        "apart, head by head": ((0, WHOLE, DIM, PAGE * DIM), (9 * WHOLE, PAGE * HEADS * v_dim, v_dim, PAGE * v_dim)),
        "side by side": ((0, 2 * WHOLE, 2 * TOKEN, 2 * DIM), (DIM, 2 * WHOLE, 2 * TOKEN, 2 * DIM)),
        "within": ((0, *thd), (0, *thd)),
        "within, head by head": ((0, WHOLE, DIM, PAGE * DIM), (0, WHOLE, DIM, PAGE * DIM)),
        "within, behind": ((0, *thd), (DIM - v_dim, *thd)),
        "one head": ((0, PAGE * DIM, DIM, 0), (9 * WHOLE, PAGE * DIM, DIM, 0)),
        "one head, within": ((0, PAGE * DIM, DIM, 0), (0, PAGE * DIM, DIM, 0)),
        "a head further": ((0, *thd), (DIM, *thd)),
    }


@pytest.mark.parametrize("type", [BF, E4, F32])
@pytest.mark.parametrize("v_dim", [64, 40])
def test_copies_into_shared_pools(draft_recorder, type, v_dim):  # noqa: F811
    kinds = _kinds(v_dim)
    group = {"within": "within", "within, head by head": "within", "within, behind": "within" if v_dim == DIM else "behind",
             "one head": "one", "one head, within": "one within", "a head further": "further"}
    for a, x in kinds.items():
        for b, y in kinds.items():
            before = draft_recorder.recorded_moves()
            rc = draft_recorder.detfold_cache_copy(_pool(ONE, *x, type, v_dim), _pool(OTHER, *y, type, v_dim), SIDE, SIDE + 64, None, 3, None)
            want = OK if b not in group or group.get(a) == group[b] else EOVERLAP
            assert rc == want, (a, b)
            assert draft_recorder.recorded_moves() == before + (rc == OK)
        c = _pool(ONE, *x, type, v_dim)
        for into in (None, c):  # within one pool all that is written twice is the same
            assert draft_recorder.detfold_cache_copy(c, into, SIDE, SIDE + 64, None, 3, None) == OK, a
