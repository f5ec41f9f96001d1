"""The decode step around the fold: a paged key-value cache, the append that
fills it, the attention of one new token over it, and the fixed-order join of
attention partials (binding of the C ABI's ``detfold_cache_append``,
``detfold_attend_paged`` and ``detfold_fold_softmax``).

    cache = PagedCache(k, v)                    [pages, page, heads, dim] views of the cache
    cache_append(cache, k, v, slots, ...)       rotate and store new tokens
    attend_paged(out, q, cache, table, lens)    one new token per row over its pages
    fold_softmax(out, outs, lses)               join the partials of W ranks, ascending

As in the rest of the package the functions only check and marshal: type,
device, shape and strides here, sizes and overlaps in the library, before
anything touches the device.  Work is enqueued on the caller's current stream
(or ``stream``); nothing synchronizes, so a call may be captured into a graph.

A call goes to ``_bind`` first, which reads the tensors in C++ and calls the
library if all is as it should be (an append with its rotation: 9.9 us a call
without it).  What it leaves comes back to the checks here, which say what is
wrong, and make the call if nothing is.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

from . import LIB_PATH, _check, _stream_handle as _stream, load as _load

F32, BF16, F16, E4M3 = 0, 1, 2, 3
ATTEND_STEP = 32
MIN_HEAD, MAX_HEAD = 16, 256

_p, _q, _i, _f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class PagedCacheC(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("pages", _q),
                ("k_page", _q), ("k_token", _q), ("k_head", _q), ("v_page", _q), ("v_token", _q),
                ("v_head", _q), ("page", _i), ("heads", _i), ("dim", _i), ("v_dim", _i), ("type", _i),
                ("reserved", _i)]


class AppendC(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("q", _p), ("q_out", _p), ("slots", _p), ("positions", _p),
                ("cos", _p), ("sin", _p), ("tokens", _q), ("angles", _q), ("k_token", _q),
                ("k_head", _q), ("v_token", _q), ("v_head", _q), ("q_token", _q), ("q_head", _q),
                ("out_token", _q), ("out_head", _q), ("type", _i), ("q_heads", _i), ("rot", _i),
                ("pairs", _i)]


class AttendC(ctypes.Structure):
    _fields_ = [("out", _p), ("q", _p), ("lse", _p), ("table", _p), ("lens", _p), ("workspace", _p),
                ("workspace_bytes", _q), ("batch", _q), ("max_len", _q), ("window", _q),
                ("table_row", _q), ("table_width", _q), ("q_row", _q), ("q_head", _q),
                ("out_row", _q), ("out_head", _q), ("scale", _f), ("type", _i), ("out_type", _i),
                ("q_heads", _i), ("split", _i), ("reserved", _i)]


class AttendPlan(ctypes.Structure):
    _fields_ = [("units", _q), ("splits", _q), ("split", _q), ("workspace_bytes", _q),
                ("workspace_upto", _q)]

    def as_dict(self) -> dict:
        return {k: getattr(self, k) for k, _ in self._fields_}


def _packer(c) -> struct.Struct:
    """One call that lays out the whole struct (a ctypes field at a time costs
    the call about 2 us)."""
    return struct.Struct("".join({_p: "P", _q: "q", _i: "i", _f: "f"}[t] for _, t in c._fields_))


_CACHE, _APPEND, _ATTEND = _packer(PagedCacheC), _packer(AppendC), _packer(AttendC)


def bind(lib) -> None:
    """Argument types of the decode-step entry points.  Structs go in as the
    bytes that the packers make."""
    i64p = ctypes.POINTER(_q)
    lib.detfold_cache_append.argtypes = [ctypes.c_char_p, ctypes.c_char_p, _p]
    lib.detfold_attend_paged.argtypes = [ctypes.c_char_p, ctypes.c_char_p, _p]
    lib.detfold_plan_attend.argtypes = [ctypes.c_char_p, _q, _i, _q, _q, _i, _i, ctypes.POINTER(AttendPlan)]
    lib.detfold_attend_workspace.argtypes = [ctypes.c_char_p, _q, _i, _q, _i, i64p]
    lib.detfold_fold_softmax.argtypes = [_p, _p, _p, _p, _i, _i, _q, _q, _q, _q, _p]


_native = None


def _bound():
    """``_bind``'s functions, each with the library's own, and torch's accessor
    of the current stream; where there is none that was built with this
    library, functions that take no call."""
    global _native
    lib = _load()
    try:
        import torch
        from . import _bind
        with open(LIB_PATH + ".sha256") as f:
            ok = f.read().strip() == _bind.built_from
        raw = torch._C._cuda_getCurrentRawStream
    except (ImportError, OSError, AttributeError):
        ok = False
    if ok:
        _native = raw, *(x for call, of in ((_bind.append, lib.detfold_cache_append),
                                            (_bind.attend, lib.detfold_attend_paged),
                                            (_bind.fold, lib.detfold_fold_softmax))
                         for x in (call, ctypes.cast(of, _p).value))
    else:
        _native = (lambda device: 0, *(lambda *args: -1, 0) * 3)
    return _native


_types = None


def _type(t, name: str) -> int:
    """The library's type of a tensor, -1 for one that it has not."""
    global _types
    if _types is None:
        import torch
        _types = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16, torch.float8_e4m3fn: E4M3}
    try:
        return _types.get(t.dtype, -1)
    except AttributeError:
        raise TypeError("%s must be a torch.Tensor" % name) from None


def _refuse_type(t, name: str, want: str) -> None:
    raise TypeError("%s must be %s, got %s" % (name, want, t.dtype))


def _heads(t, name: str, dev: int, heads, dim: int):
    """Strides of a [n, heads, dim] view with contiguous heads."""
    if t.dim() != 3 or t.shape[2] != dim or (heads and t.shape[1] != heads):
        raise ValueError("%s must be [n, %s, %d], got %s" % (name, heads or "heads", dim, tuple(t.shape)))
    return _place(t, name, dev)


def _place(t, name: str, dev: int):
    if t.get_device() != dev:
        raise ValueError("%s must be on the cache's device, got %s" % (name, t.device))
    s = t.stride()
    if s[-1] != 1 and t.shape[-1] > 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    return s


def _plain(t, name: str, dev: int, dtype: str, shape) -> int:
    """The address of a contiguous tensor of a shape and type ('int32', ...)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != getattr(torch, dtype):
        _refuse_type(t, name, dtype)
    if t.get_device() != dev:
        raise ValueError("%s must be on the cache's device, got %s" % (name, t.device))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


class PagedCache:
    """A paged key-value cache: two tensors ``k`` [pages, page, heads, dim] and
    ``v`` [pages, page, heads, v_dim], views that may lie token-major or
    head-major in memory (a head's values are contiguous).  Slot ``s`` is token
    ``s % page`` of page ``s // page``.  An 8-bit cache (``float8_e4m3fn``) may
    have ``k_scale`` and ``v_scale``, a float32 per head: a stored value stands
    for value * scale.  The object keeps the tensors and describes them to the
    library once; they must not be resized while it is in use."""

    def __init__(self, k, v, *, k_scale=None, v_scale=None):
        type_ = _type(k, "k")
        if type_ < 0:
            _refuse_type(k, "k", "float32, bfloat16, float16 or float8_e4m3fn")
        if _type(v, "v") != type_:
            _refuse_type(v, "v", "of k's type, %s" % k.dtype)
        if k.device.type != "cuda":
            raise ValueError("k must be a device tensor, got %s" % k.device)
        if k.dim() != 4 or v.dim() != 4 or v.shape[:3] != k.shape[:3]:
            raise ValueError("k and v must be [pages, page, heads, dim], got %s and %s"
                             % (tuple(k.shape), tuple(v.shape)))
        pages, page, heads, dim = k.shape
        dev = k.get_device()
        for x, nm in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if x is not None and type_ != E4M3:
                raise ValueError("%s is for float8_e4m3fn caches" % nm)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.page, self.heads, self.dim, self.v_dim = pages, page, heads, dim, v.shape[3]
        self.type, self.device_index = type_, dev
        self._c = self._described()

    def _described(self) -> bytes:
        """The cache for the library, where its tensors lie now."""
        k, v, dev = self.k, self.v, self.device_index
        for x, nm, dim in ((k, "k", self.dim), (v, "v", self.v_dim)):
            if tuple(x.shape) != (self.pages, self.page, self.heads, dim) or _type(x, nm) != self.type:
                raise ValueError("the cache's %s has changed its shape or type, to %s of %s" % (nm, tuple(x.shape), x.dtype))
        ks, vs = _place(k, "k", dev), _place(v, "v", dev)
        scales = [0 if x is None else _plain(x, nm, dev, "float32", (self.heads,))
                  for x, nm in ((self.k_scale, "k_scale"), (self.v_scale, "v_scale"))]
        return _CACHE.pack(k.data_ptr(), v.data_ptr(), scales[0], scales[1], self.pages, ks[0], ks[1], ks[2],
                           vs[0], vs[1], vs[2], self.page, self.heads, self.dim, self.v_dim, self.type, 0)


def _same(t, name: str, want: int, like) -> None:
    if _type(t, name) != want:
        _refuse_type(t, name, "of the same type as %s" % like)


def cache_append(cache: PagedCache, k, v, slots, *, q=None, q_out=None, positions=None, cos=None, sin=None,
                 pairs: bool = False, stream=None) -> None:
    """Write ``k`` [tokens, heads, dim] and ``v`` [tokens, heads, v_dim] into the
    cache at ``slots`` (int64; negative or past the cache: not stored).

    With ``cos`` and ``sin`` (float32 [angles, rot / 2]) the first ``rot``
    values of every key head, and of every head of ``q`` [tokens, q_heads, dim]
    into ``q_out``, turn by the angles of the token's ``positions`` (int64):
    value i with i + rot / 2, or with ``pairs`` 2i with 2i + 1.  ``q_out`` may
    be ``q``.  The tensors may be strided views of one projection; tokens of
    one call must not share a slot."""
    dev = cache.device_index
    current, call, of = (_native or _bound())[:3]
    rc = call(of, cache, dev, current(dev) if stream is None else int(stream.cuda_stream), k, v, slots, q, q_out,
              positions, cos, sin, pairs)
    if rc >= 0:
        return _check(rc, "cache_append") if rc else None
    type_ = _type(k, "k")
    _same(v, "v", type_, "k")
    ks, vs = _heads(k, "k", dev, cache.heads, cache.dim), _heads(v, "v", dev, cache.heads, cache.v_dim)
    tokens = k.shape[0]
    if v.shape[0] != tokens:
        raise ValueError("k has %d tokens, v %d" % (tokens, v.shape[0]))
    qp = op = q_heads = 0
    qs = os = (0, 0)
    if q is not None:
        if q_out is None:
            raise ValueError("q needs q_out")
        _same(q, "q", type_, "k")
        _same(q_out, "q_out", type_, "k")
        q_heads = q.shape[1] if q.dim() == 3 else 0
        qs, os = _heads(q, "q", dev, q_heads, cache.dim), _heads(q_out, "q_out", dev, q_heads, cache.dim)
        if q.shape[0] != tokens or q_out.shape[0] != tokens:
            raise ValueError("k has %d tokens, q %d and q_out %d" % (tokens, q.shape[0], q_out.shape[0]))
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    pp = cp = sp = rot = angles = 0
    if cos is not None or sin is not None:
        if cos is None or sin is None or positions is None:
            raise ValueError("the rotation needs positions, cos and sin")
        if cos.dim() != 2:
            raise ValueError("cos must be [angles, rot / 2], got %s" % (tuple(cos.shape),))
        angles, half = cos.shape
        rot = 2 * half
        cp, sp = _plain(cos, "cos", dev, "float32", (angles, half)), _plain(sin, "sin", dev, "float32", (angles, half))
        pp = _plain(positions, "positions", dev, "int64", (tokens,))
    elif positions is not None:
        raise ValueError("positions need cos and sin")
    args = _APPEND.pack(k.data_ptr(), v.data_ptr(), qp, op, _plain(slots, "slots", dev, "int64", (tokens,)), pp,
                        cp, sp, tokens, angles, ks[0], ks[1], vs[0], vs[1], qs[0], qs[1], os[0], os[1], type_,
                        q_heads, rot, 1 if pairs else 0)
    _check(_load().detfold_cache_append(cache._described(), args, _stream(k, stream)), "cache_append")


def _within(stream, dev: int):
    """The context in which torch allocates for `stream` (None: the current one)."""
    import torch
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(int(stream.cuda_stream), device=dev))


def attend_workspace(cache: PagedCache, batch: int, q_heads: int, max_len: int, *, split: int = 0):
    """The device memory that ``attend_paged`` joins the parts of long rows in,
    for calls whose batch and ``max_len`` are at most these (a uint8 tensor).
    Calls that overlap in time must not share one.  It is allocated on torch's
    current stream: for calls on another one, make it within that
    (``torch.cuda.stream``), or keep it until they are done."""
    import torch
    n = ctypes.c_int64()
    _check(_load().detfold_attend_workspace(cache._c, batch, q_heads, max_len, split, ctypes.byref(n)),
           "attend_workspace")
    return torch.empty(n.value, dtype=torch.uint8, device=cache.k.device)


def attend_paged(out, q, cache: PagedCache, table, lens, *, scale=None, window: int = 0, max_len=None, lse=None,
                 workspace=None, split: int = 0, stream=None) -> None:
    """Attention of one new token per row: ``out`` [batch, q_heads, v_dim] and,
    where given, ``lse`` [batch, q_heads] (float32) of ``q`` [batch, q_heads,
    dim] over the first ``lens`` (int32) tokens of each row, whose pages
    ``table`` (int32 [batch, width]) names.

    ``scale`` defaults to 1 / sqrt(dim); with ``window`` a row sees its last
    ``window`` tokens only.  ``max_len``, a bound of ``lens`` known on the host,
    sizes the launch (default: all that the table can name).  A row without a
    token gives 0 and -infinity; a length or page out of range gives NaN.
    ``out`` is of q's type or float32.  ``workspace`` is ``attend_workspace``'s
    (allocated for the call where it is missing).  ``split`` fixes the tokens
    of one part (a multiple of 32), so that a row's bits do not depend on the
    batch around it."""
    dev = cache.device_index
    current, _, _, call, of = (_native or _bound())[:5]
    rc = call(of, cache, dev, current(dev) if stream is None else int(stream.cuda_stream), out, q, table, lens,
              1.0 / math.sqrt(cache.dim) if scale is None else scale, window, max_len, lse, workspace, split)
    if rc >= 0:
        return _check(rc, "attend_paged") if rc else None
    type_, out_type = _type(q, "q"), _type(out, "out")
    if out_type != type_ and out_type != F32:
        _refuse_type(out, "out", "of q's type or float32")
    if q.dim() != 3:
        raise ValueError("q must be [batch, q_heads, %d], got %s" % (cache.dim, tuple(q.shape)))
    batch, q_heads = q.shape[0], q.shape[1]
    qs, os = _heads(q, "q", dev, q_heads, cache.dim), _heads(out, "out", dev, q_heads, cache.v_dim)
    if out.shape[0] != batch:
        raise ValueError("q has %d rows, out %d" % (batch, out.shape[0]))
    lens_p = _plain(lens, "lens", dev, "int32", (batch,))
    if _type(table, "table") >= 0 or str(table.dtype) != "torch.int32":
        _refuse_type(table, "table", "int32")
    if table.dim() != 2 or table.shape[0] != batch:
        raise ValueError("table must be [%d, width], got %s" % (batch, tuple(table.shape)))
    ts, width = _place(table, "table", dev), table.shape[1]
    lse_p = 0 if lse is None else _plain(lse, "lse", dev, "float32", (batch, q_heads))
    if max_len is None:
        max_len = min(width * cache.page, 2 ** 31 - 1)
    if workspace is None:
        # In the pool of the stream that uses it: what this call frees on return
        # goes to no other stream before the parts are joined.
        with _within(stream, dev):
            workspace = attend_workspace(cache, batch, q_heads, max_len, split=split)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    args = _ATTEND.pack(out.data_ptr(), q.data_ptr(), lse_p, table.data_ptr(), lens_p, workspace.data_ptr(),
                        workspace.nbytes, batch, max_len, window, ts[0], width, qs[0], qs[1], os[0], os[1],
                        1.0 / math.sqrt(cache.dim) if scale is None else scale, type_, out_type, q_heads, split, 0)
    _check(_load().detfold_attend_paged(cache._described(), args, _stream(q, stream)), "attend_paged")


def plan_attend(cache, batch: int, q_heads: int, max_len: int, cu_count: int, *, window: int = 0,
                split: int = 0) -> dict:
    """How ``attend_paged`` would split such a call (host only): ``cache`` is a
    ``PagedCache`` or the bytes of a ``PagedCacheC``."""
    p = AttendPlan()
    _check(_load().detfold_plan_attend(cache._c if isinstance(cache, PagedCache) else bytes(cache), batch, q_heads,
                                       max_len, window, split, cu_count, ctypes.byref(p)), "plan_attend")
    return p.as_dict()


def fold_softmax(out, outs, lses, *, lse=None, stream=None) -> None:
    """The fixed-order join of W attention partials: ``outs`` [W, ..., dim] (float32,
    bfloat16 or float16), each the mean of its own tokens under softmax, with
    ``lses`` [W, ...] (float32) the logarithms of their sums of exponentials,
    into ``out`` [..., dim] and, where given, ``lse`` [...].

    A partial with ``lses`` = -infinity had no token and adds nothing, whatever
    its ``outs`` hold.  The partials may be padded apart; each is contiguous."""
    type_ = _type(outs, "outs")
    dev = outs.get_device()
    native = _native or _bound()
    if dev >= 0:
        rc = native[5](native[6], dev, native[0](dev) if stream is None else int(stream.cuda_stream), out, outs, lses, lse)
        if rc >= 0:
            return _check(rc, "fold_softmax") if rc else None
    _same(out, "out", type_, "outs")
    if dev < 0:
        raise ValueError("outs must be a device tensor, got %s" % outs.device)
    if outs.dim() < 2 or outs.shape[0] < 1:
        raise ValueError("outs must be [W, ..., dim], got %s" % (tuple(outs.shape),))
    W, dim = outs.shape[0], outs.shape[-1]
    rows = outs.shape[1:-1].numel()
    if tuple(lses.shape) != tuple(outs.shape[:-1]):
        raise ValueError("lses must have shape %s, got %s" % (tuple(outs.shape[:-1]), tuple(lses.shape)))
    if out.shape != outs.shape[1:] or out.get_device() != dev or not out.is_contiguous():
        raise ValueError("out must be contiguous, %s, on the device of outs" % (tuple(outs.shape[1:]),))
    _same(lses, "lses", F32, "float32")
    if lses.get_device() != dev:
        raise ValueError("lses must be on the device of outs, got %s" % lses.device)
    if not outs[0].is_contiguous() or not lses[0].is_contiguous():
        raise ValueError("each partial of outs and lses must be contiguous")
    lse_p = 0 if lse is None else _plain(lse, "lse", dev, "float32", outs.shape[1:-1])
    _check(_load().detfold_fold_softmax(out.data_ptr(), outs.data_ptr(), lses.data_ptr(), lse_p, type_, W, rows, dim,
                                        outs.stride(0) if W > 1 else rows * dim, lses.stride(0) if W > 1 else rows,
                                        _stream(outs, stream)), "fold_softmax")
