"""Where the binding's own allocation of a call lies (CPU only; the library's
entry and the stream context are stood in for)."""
import contextlib
import types

import pytest
import torch

from deterministic_fixed_order_amd import decode as d


class Library:
    def __init__(self):
        self.calls = []

    def detfold_attend_paged(self, cache, args, stream):
        self.calls.append((d._ATTEND.unpack(args), stream))
        return 0


@pytest.fixture
def stood_in(monkeypatch):
    """attend_paged on host tensors: what it enqueues, and the streams that were
    current when a workspace was made."""
    lib, current, made = Library(), [0], []
    handle = lambda s: 0 if s is None else int(s.cuda_stream)  # noqa: E731

    @contextlib.contextmanager
    def stream_context(s):
        current.append(current[-1] if s is None else handle(s))
        yield
        current.pop()

    def workspace(cache, batch, q_heads, max_len, *, split=0):
        made.append(current[-1])
        return torch.empty(1 << 12, dtype=torch.uint8)

    monkeypatch.setattr(d, "_native", (lambda dev: 0, *(lambda *a: -1, 0) * 3))
    monkeypatch.setattr(d, "_load", lambda: lib)
    monkeypatch.setattr(d, "_stream", lambda t, s: handle(s))
    monkeypatch.setattr(d, "attend_workspace", workspace)
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: types.SimpleNamespace(cuda_stream=h))
    cache = object.__new__(d.PagedCache)
    cache.k = cache.v = torch.zeros((4, 16, 2, 64))
    cache.k_scale = cache.v_scale = None
    cache.device_index, cache.heads, cache.dim, cache.v_dim, cache.page, cache.pages, cache.type = -1, 2, 64, 64, 16, 4, d.F32
    q = torch.zeros((3, 4, 64))

    def call(**kw):
        d.attend_paged(torch.empty_like(q), q, cache, torch.zeros((3, 4), dtype=torch.int32),
                       torch.zeros(3, dtype=torch.int32), **kw)
        return lib.calls[-1], made
    return call


def test_a_call_on_another_stream_has_its_workspace_from_there(stood_in):
    """Freed to the current stream's pool, it would be written again while the
    other stream still joins the parts in it."""
    (args, stream), made = stood_in(stream=types.SimpleNamespace(cuda_stream=77))
    assert stream == 77 and made == [77]


def test_a_call_on_the_current_stream(stood_in):
    (args, stream), made = stood_in()
    assert stream == 0 and made == [0]


def test_the_callers_workspace_is_taken(stood_in):
    mine = torch.empty(4096, dtype=torch.uint8)
    (args, stream), made = stood_in(stream=types.SimpleNamespace(cuda_stream=77), workspace=mine)
    assert made == [] and mine.data_ptr() in args and stream == 77
