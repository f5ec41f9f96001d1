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


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("tokens,q_heads,heads,dim,v_dim,rot", [
    (9, 15, 3, 84, 84, 28), (9, 5, 1, 66, 33, 66), (9, 6, 3, 250, 246, 124), (9, 2, 1, 18, 22, 2), (9, 4, 2, 80, 64, 40),
    (9, 3, 3, 96, 96, 96), (9, 8, 8, 192, 128, 0), (9, 2, 2, 17, 19, 0)])
def test_in_place_where_accesses_narrow(env, dtype, cache, pairs, tokens, q_heads, heads, dim, v_dim, rot):  # noqa: F811
    _append_case(env, tokens, q_heads, heads, dim, v_dim, dtype, cache, 7, rot, pairs, in_place=True, idle=(2, 5))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,cache,q_heads,heads,dim,v_dim,rot,pairs", [
    ("bf16", "bf16", 15, 3, 84, 84, 28, True), ("f32", "e4m3", 5, 1, 66, 33, 66, False), ("f16", "f16", 7, 5, 128, 128, 128, False),
    ("f32", "bf16", 6, 3, 250, 246, 124, False), ("bf16", "e4m3", 9, 9, 64, 64, 64, True)])
def test_two_heads_a_thread(env, in_place, dtype, cache, q_heads, heads, dim, v_dim, rot, pairs):  # noqa: F811
    """Enough tokens that a thread takes two heads; odd counts of them leave one over."""
    width = 16 // (4 if dtype == "f32" else 2)
    tokens = -(-(1 << 20) // ((q_heads + heads) * (dim // width)))
    _append_case(env, tokens, q_heads, heads, dim, v_dim, dtype, cache, 16, rot, pairs, in_place=in_place, idle=(3, tokens - 2))
