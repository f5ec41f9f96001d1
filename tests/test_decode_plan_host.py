"""The attention's plan over extreme sizes (CPU only): accepted plans cover the
tokens and keep their byte counts in range, others are refused."""
import ctypes
import random

from test_decode_host import attend, cache, lib  # noqa: F401

from deterministic_fixed_order_amd import EDEVICE, EINVAL
from deterministic_fixed_order_amd import decode as d


def test_extreme_plans(lib):  # noqa: F811
    rng = random.Random(12)

    def size(top):
        return rng.choice([0, 1, 2, top, top - 1, rng.randint(0, top), int(2 ** rng.uniform(0, top.bit_length())) % (top + 1)])
    accepted = 0
    for _ in range(20000):
        heads = max(1, size(1 << 16))
        group = max(1, size((1 << 16) // heads))
        dim = rng.randint(16, 256)
        c = cache(heads=heads, dim=dim, v_dim=rng.randint(16, 256), k_head=256, v_head=256, k_token=256 * heads,
                  v_token=256 * heads, k_page=256 * heads * 16, v_page=256 * heads * 16)
        batch, max_len, window = size((1 << 31) - 1), size((1 << 31) - 1), rng.choice([0, size((1 << 31) - 1)])
        split, cu = rng.choice([0, 0, 32, 32 * size(1 << 24)]), rng.choice([1, 2, 7, 64, 256, 304, 1 << 20])
        p = d.AttendPlan()
        rc = lib.detfold_plan_attend(c, batch, heads * group, max_len, window, split, cu, ctypes.byref(p))
        assert rc in (0, 1)
        if rc:
            continue
        accepted += 1
        seen = min(window, max_len) if window else max_len
        assert p.splits >= 1 and p.splits * p.split >= seen and 0 <= p.workspace_bytes <= p.workspace_upto < 1 << 62
        assert p.units == batch * heads * -(-group // 16)
    assert accepted > 5000


def test_a_row_in_too_many_parts_is_refused(lib):  # noqa: F811
    """Every other argument is in order; 2^26 parts of one row are not launched."""
    got = lib.detfold_attend_paged(cache(), attend(batch=1, max_len=(1 << 31) - 1, split=32), None)
    assert got in (EINVAL, EDEVICE)  # EDEVICE: no device to plan for, and nothing is launched either
