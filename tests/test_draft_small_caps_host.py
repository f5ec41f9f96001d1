"""Caps that are not 0 but would be in binary32, where 0 is no cap (CPU only): the C++ side of
the call leaves them to the Python side, and that refuses them."""
from test_decode_binding_host import _run

CALL = """
import types
from deterministic_fixed_order_amd import draft

TREE = ctypes.CFUNCTYPE(ctypes.c_int, P, P, P)(lambda c, a, s: (seen.append(draft.TreeC.from_buffer_copy(
    ctypes.string_at(a, ctypes.sizeof(draft.TreeC))).cap), 7)[1])


def tree(cap, dims):
    q = torch.ones((3, 2, 4, 64)[:1] + (3, 2, 4, 64)[5 - dims:])
    table, lens = torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    return _bind.tree(at(TREE), Cache("cpu"), -1, 0, torch.empty_like(q), q, table, lens, None, None, None, cap, None, 0.125, 0, 64, None,
                      torch.empty(64), 0, dims)


def python(cap):
    c = types.SimpleNamespace(device_index=-1, dim=64, v_dim=64, page=16, type=d.F32, k=torch.zeros(1))
    q = torch.ones((3, 2, 4, 64))
    draft._attend("attend_tree", torch.empty_like(q), q, c, torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32), None,
                  None, None, cap, None, None, 0, 64, None, torch.empty(64), 0, None)


for dims in (3, 4):
    for cap in (0.0, -0.0, 0, 30, 30.0, 1e-37, 2.0 ** -126, 2.0 ** 127):
        assert tree(cap, dims) == 7, cap
        assert seen.pop() == ctypes.c_float(cap).value
    for cap in (1e-50, -1e-50, 1e-46, 5e-324, -5e-324):
        assert tree(cap, dims) == -1, cap
        try:
            python(cap)
            print("taken")
        except ValueError as e:
            assert "cap" in str(e)
assert not seen
print("refused")
"""


def test_caps_that_binary32_has_not():
    assert _run(CALL) == "refused"
