"""A workspace of some sizes serves every smaller call (CPU only): over caches of every type,
values of another size than the keys, and layouts that workgroups do and do not stage."""
import ctypes
import random

import pytest

from deterministic_fixed_order_amd import decode as d
from test_decode_host import BF, E4, F16, F32, cache, lib  # noqa: F401

TYPES = {BF: [BF, F32], F16: [F16], F32: [F32], E4: [BF, F16, F32]}


def _plan(lib, c, batch, drafts, q_heads, max_len, window, split, type, out, cu):  # noqa: F811
    p = d.AttendPlan()
    assert lib.detfold_plan_tree(c, batch, drafts, q_heads, max_len, window, split, type, out, cu, ctypes.byref(p)) == 0
    return p


@pytest.mark.parametrize("kind", [BF, F16, F32, E4])
@pytest.mark.parametrize("seed", range(4))
def test_workspaces_serve_smaller_calls(lib, kind, seed):  # noqa: F811
    rng = random.Random(100 * kind + seed)
    for _ in range(120):
        heads, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 4, 5, 8, 16, 24])
        dim = rng.choice([16, 64, 80, 128, 192, 256, rng.randint(16, 256)])
        v_dim = rng.choice([dim, dim, 64, 128, rng.randint(16, 256)])
        page, gap = rng.choice([1, 7, 16, 64]), rng.choice([0, 0, 1, 8])
        kt, vt = heads * dim + gap, heads * v_dim + gap
        c = cache(type=kind, heads=heads, dim=dim, v_dim=v_dim, page=page, pages=50, k_head=dim, k_token=kt, k_page=page * kt, v_head=v_dim,
                  v_token=vt, v_page=page * vt)
        batch, drafts, cu = rng.choice([1, rng.randint(1, 300), 6000]), rng.randint(1, 64), rng.choice([1, 64, 256, 304])
        max_len, split = rng.choice([rng.randint(1, 3000), rng.randint(1, 200000)]), rng.choice([0, 0, 0, 64, 2048])
        if split and batch * heads * group * drafts * max_len // split > 1 << 38:
            continue
        made_for = F16 if kind == F16 else F32  # as detfold_tree_workspace asks
        most = _plan(lib, c, batch, drafts, heads * group, max_len, 0, split, made_for, made_for, cu).workspace_upto
        plain = d.AttendPlan()
        assert lib.detfold_plan_attend(c, batch, heads * group, max_len, 0, split, cu, ctypes.byref(plain)) == 0
        for _ in range(30):
            b, n = rng.randint(0, batch), min(max_len, rng.choice([max_len, rng.randint(0, max_len), rng.randint(0, 400)]))
            t, w, type = rng.randint(1, drafts), rng.choice([0, rng.randint(1, 5000)]), rng.choice(TYPES[kind])
            out = rng.choice([type, F32])
            p = _plan(lib, c, b, t, heads * group, n, w, split, type, out, cu)
            assert p.workspace_bytes <= p.workspace_upto <= most, (batch, drafts, max_len, split, b, t, n, w)
            one = _plan(lib, c, b, 1, heads * group, n, w, split, type, out, cu)
            assert one.workspace_bytes <= plain.workspace_upto, (batch, max_len, split, b, n, w)
