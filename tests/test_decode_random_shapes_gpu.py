"""The decode-step operators on seeded random shapes: types, head counts and sizes,
page sizes and orders, lengths, windows, splits and rotations together, against
their 64-bit forms."""
import random

import pytest

from test_decode_gpu import PAIRS, _append_case, _attend_case, _fold_case, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _log(rng, low, high):
    return max(low, min(high, int(low * (high / low) ** rng.random())))


def _heads(rng):
    heads = rng.choice([1, 1, 2, 3, 4, 5, 8, 12])
    dim = rng.choice([64, 128, 256, rng.randint(16, 256), rng.randint(16, 256), 16 * rng.randint(1, 16)])
    return heads, dim, rng.choice([dim, dim, rng.randint(16, 256)])


@pytest.mark.parametrize("seed", range(160))
def test_attend(env, seed):  # noqa: F811
    rng = random.Random(seed)
    heads, dim, v_dim = _heads(rng)
    q_heads = heads * rng.choice([1, 1, 2, 3, 4, 7, 8, 16, 17, 24, 40])
    (dtype, cache), page = rng.choice(PAIRS), rng.choice([1, 2, 5, 7, 16, 16, 32, 48, 64, 100, 256])
    rows = _log(rng, 1, 40)
    longest = _log(rng, 1, max(2, 2000000 // (rows * heads * (dim + v_dim))) + 40)
    lens = [rng.choice([0, rng.randint(0, longest), longest, _log(rng, 1, longest)]) for _ in range(rows)]
    window, split = rng.choice([0, 0, 0, _log(rng, 1, longest + 5)]), rng.choice([0, 0, 0, 32, 64, 32 * rng.randint(1, 40)])
    out, scale = rng.choice([None, None, "f32"]), rng.choice([None, None, None, -0.2, 0.05])
    case = (seed, lens, q_heads, heads, dim, v_dim, dtype, cache, page, window, split, out, scale)
    _attend_case(env, lens, q_heads, heads, dim, v_dim, dtype, cache, page, rng.choice(["thd", "htd"]), window=window, out=out,
                 scale=scale, split=split, spread=rng.choice([1.0, 1.0, 4.0]), say=case)


@pytest.mark.parametrize("seed", range(120))
def test_append(env, seed):  # noqa: F811
    rng = random.Random(seed)
    heads, dim, v_dim = _heads(rng)
    q_heads = heads * rng.choice([0, 1, 2, 4, 7])
    (dtype, cache), page, tokens = rng.choice(PAIRS), rng.choice([1, 3, 7, 16, 64]), _log(rng, 1, 400)
    rot = rng.choice([0, dim // 2 * 2, 2 * rng.randint(0, dim // 2)])
    idle = [i for i in range(tokens) if rng.random() < 0.2]
    print("case: append", (seed, tokens, q_heads, heads, dim, v_dim, dtype, cache, page, rot), flush=True)
    _append_case(env, tokens, q_heads, heads, dim, v_dim, dtype, cache, page, rot, rng.random() < 0.5,
                 rng.choice(["thd", "htd", "pair"]), idle=idle, in_place=q_heads > 0 and rng.random() < 0.4)


@pytest.mark.parametrize("seed", range(80))
def test_fold(env, seed):  # noqa: F811
    rng = random.Random(seed)
    W, dim = _log(rng, 1, 70), rng.choice([1, 64, 128, rng.randint(1, 300), rng.randint(1, 40)])
    rows = _log(rng, 1, max(2, 400000 // (W * dim)))
    print("case: fold", (seed, W, rows, dim), flush=True)
    _fold_case(env, W, (rows,), dim, rng.choice(["f32", "bf16", "f16"]), empty=rng.choice([0.0, 0.3, 0.9]),
               pad=rng.randint(0, 9), spread=rng.choice([1.0, 3.0, 40.0]))
