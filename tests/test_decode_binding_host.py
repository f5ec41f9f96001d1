"""The C++ side of the decode step's Python calls (CPU only): what it takes, it
hands on as it is; what it cannot read, it leaves to the Python side, and no C++
exception ends the process.  The library's entry is stood in for by a recorder,
and the device tensors have no memory (fake tensors) or are the host's."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PREAMBLE = """
import ctypes, sys
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import deterministic_fixed_order_amd
from deterministic_fixed_order_amd import _bind, decode as d

seen = []
P, I, Q = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
STRUCT = ctypes.CFUNCTYPE(ctypes.c_int, P, P, P)(lambda c, a, s: (seen.append(d.PagedCacheC.from_buffer_copy(
    ctypes.string_at(c, ctypes.sizeof(d.PagedCacheC)))), 7)[1])
FOLD = ctypes.CFUNCTYPE(ctypes.c_int, P, P, P, P, I, I, Q, Q, Q, Q, P)(lambda *a: (seen.append(a), 7)[1])
at = lambda f: ctypes.cast(f, P).value


class Cache:
    # what the binding reads of a PagedCache
    _c = bytes(d.PagedCacheC(k=1 << 40, v=1 << 41, pages=4, k_page=2048, k_token=128, k_head=64, v_page=2048, v_token=128,
                             v_head=64, page=16, heads=2, dim=64, v_dim=64, type=d.F32))

    def __init__(self, device):
        self.k, self.v = (torch.zeros((4, 16, 2, 64), device=device) for _ in range(2))


def append(x, q, dev):
    n = x.shape[0]
    return _bind.append(at(STRUCT), Cache(q.device), dev, 0, x, x, torch.zeros(n, dtype=torch.int64, device=x.device), q, q, None,
                        None, None, False)


def attend(x, q, dev):
    n = q.shape[0]
    table, lens = (torch.zeros(s, dtype=torch.int32, device=q.device) for s in ((n, 4), (n,)))
    return _bind.attend(at(STRUCT), Cache(q.device), dev, 0, torch.empty_like(q), q, table, lens, 0.125, 0, 64, None,
                        torch.empty(64, device=q.device), 0)


def fold(x, q, dev):
    return _bind.fold(at(FOLD), dev, 0, q[0], q, q[..., 0].contiguous(), None)
"""

TRANSFORMS = """
class Done(Exception):
    "The call is made; the transform itself needs a device to go on."


op = {"append": append, "attend": attend, "fold": fold}[sys.argv[1]]
with FakeTensorMode():
    x, q = torch.ones((3, 2, 64), device="cuda"), torch.ones((3, 4, 64), device="cuda")
    got = []

    def f(x, q):
        got.append(op(x, q, 0))
        raise Done
    try:
        if sys.argv[2] == "vmap":
            torch.func.vmap(f)(torch.ones((5, 3, 2, 64), device="cuda"), torch.ones((5, 3, 4, 64), device="cuda"))
        elif sys.argv[2] == "grad":
            torch.func.grad(f, (0, 1))(x, q)
        else:
            torch.func.jvp(f, (x, q), (x, q))
    except Done:
        pass
assert got == [-1] and not seen, (got, seen)
print("left to python")
"""


def _run(text, *args):
    res = subprocess.run([sys.executable, "-c", PREAMBLE + text, *args], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert res.returncode == 0, "exit %d\n%s" % (res.returncode, res.stderr[-3000:])
    return res.stdout.strip()


@pytest.mark.parametrize("op", ["append", "attend", "fold"])
@pytest.mark.parametrize("transform", ["vmap", "grad", "jvp"])
def test_wrapped_tensors_are_left_to_python(op, transform):
    """A tensor inside a function transform has no address: asking for it throws."""
    assert _run(TRANSFORMS, op, transform) == "left to python"


def test_what_is_in_order_is_handed_on():
    assert _run("""
x, q = torch.ones((3, 2, 64)), torch.ones((3, 4, 64))
assert append(x, q, -1) == 7 and attend(x, q, -1) == 7
with FakeTensorMode():
    assert fold(None, torch.ones((3, 4, 64), device="cuda"), 0) == 7
assert len(seen) == 3
print("handed on")
""") == "handed on"


@pytest.mark.parametrize("transform", ["vmap", "grad", "jvp"])
def test_python_refuses_wrapped_tensors(transform):
    """The checks that take over raise an ordinary error."""
    assert _run("""
import types
with FakeTensorMode():
    def f(q):
        d.fold_softmax(q[0], q, q[..., 0].contiguous(), stream=types.SimpleNamespace(cuda_stream=0))
        return q.sum()
    q = torch.ones((3, 4, 64), device="cuda")
    try:
        {"vmap": lambda: torch.func.vmap(f)(torch.ones((5, 3, 4, 64), device="cuda")), "grad": lambda: torch.func.grad(f)(q),
         "jvp": lambda: torch.func.jvp(f, (q,), (q,))}[sys.argv[1]]()
    except RuntimeError as e:
        print("refused")
""", transform) == "refused"


def test_the_caches_memory_is_read_at_each_call():
    """Other memory, other strides, another shape; and a lazy copy of a cache that is appended to."""
    assert _run("""
x, q, c = torch.ones((3, 2, 64)), torch.ones((3, 4, 64)), Cache("cpu")
Cache = lambda device: c
for step in range(4):
    for op in (append, attend):
        got = op(x, q, -1)
        assert got == (7 if step < 3 else -1), (step, op, got)
        if got == 7:
            s = seen.pop()
            assert (s.k, s.v) == (c.k.data_ptr(), c.v.data_ptr())
            assert (s.k_page, s.k_token, s.k_head) == c.k.stride()[:3] and (s.v_page, s.v_token, s.v_head) == c.v.stride()[:3]
    if step == 0:
        c.k.data, c.v.data = torch.zeros((4, 16, 2, 64)), torch.zeros((4, 2, 16, 64)).transpose(1, 2)
    elif step == 1:
        lazy = torch._lazy_clone(c.k)
    elif step == 2:
        c.v.data = torch.zeros((3, 16, 2, 64))
lazy_address = torch._C._data_address(lazy)
assert lazy_address != c.k.data_ptr()
print("read")
""") == "read"
