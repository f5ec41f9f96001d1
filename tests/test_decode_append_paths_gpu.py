"""Forms of ``cache_append`` that take their own path: keys and values without
queries, and queries turned in place at sizes where an access must divide its
run, with one head a thread and with two."""
import pytest

from test_decode_gpu import PAIRS, _append_case, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("heads,dim,v_dim,rot,pairs,order", [
    (1, 17, 17, 0, False, "thd"), (3, 84, 84, 28, True, "thd"), (2, 84, 80, 84, False, "htd"), (3, 250, 246, 124, False, "htd"),
    (1, 66, 33, 66, True, "thd"), (4, 128, 128, 128, False, "thd"), (5, 19, 21, 2, True, "htd")])
def test_keys_without_queries(env, dtype, cache, heads, dim, v_dim, rot, pairs, order):  # noqa: F811
    _append_case(env, 13, 0, heads, dim, v_dim, dtype, cache, 7, rot, pairs, order, idle=(2, 3, 4, 9))
