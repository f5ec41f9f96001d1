"""The access width of an append (CPU only, launches recorded): 16 bytes wherever
each run of values holds that many, and narrower only where queries turn in
place, whose runs it must divide."""
import pytest

from decode_recorder import recorder  # noqa: F401
from test_decode_host import BF, F32, Q, append, cache

NEVER = dict(q=0, q_out=0, q_heads=0)
IN_PLACE = dict(q_out=Q + (1 << 31))


def _width(lib, dim, v_dim, rot, type, **kw):
    c = cache(heads=1, dim=dim, v_dim=v_dim, k_head=dim, k_token=dim, k_page=16 * dim, v_head=v_dim, v_token=v_dim,
              v_page=16 * v_dim, type=type)
    a = append(type=type, rot=rot, k_token=dim, k_head=dim, v_token=v_dim, v_head=v_dim, **{
        **dict(q_heads=1, q_token=dim, q_head=dim, out_token=dim, out_head=dim), **kw})
    assert lib.detfold_cache_append(c, a, None) == 0
    return lib.recorded_width()


@pytest.mark.parametrize("type,most", [(BF, 8), (F32, 4)])
@pytest.mark.parametrize("queries", [{}, NEVER], ids=["queries", "no queries"])
def test_runs_of_any_size_take_whole_accesses(recorder, queries, type, most):  # noqa: F811
    for dim, v_dim, rot in ((128, 128, 128), (17, 17, 0), (84, 84, 0), (84, 84, 28), (250, 246, 124), (66, 33, 66), (19, 21, 0)):
        assert _width(recorder, dim, v_dim, rot, type, **queries) == most, (dim, v_dim, rot)


@pytest.mark.parametrize("queries", [{}, NEVER], ids=["queries", "no queries"])
def test_short_runs_hold_one_access(recorder, queries):  # noqa: F811
    for rot, width in ((2, 1), (4, 2), (6, 2), (8, 4), (16, 8)):
        assert _width(recorder, 64, 64, rot, BF, **queries) == width
    assert _width(recorder, 20, 64, 16, BF, **queries) == 4


def test_in_place_divides_its_runs(recorder):  # noqa: F811
    for dim, v_dim, rot, width in ((128, 128, 128, 8), (84, 84, 28, 2), (66, 66, 66, 1), (250, 246, 124, 2), (64, 64, 32, 8), (84, 84, 0, 4)):
        assert _width(recorder, dim, v_dim, rot, BF, **IN_PLACE) == width, (dim, v_dim, rot)
