"""The drafted step: several new tokens of a row at once, of which some are kept
(binding of the C ABI's ``detfold_attend_tree``, ``detfold_cache_copy`` and
``detfold_cache_compact``).

    cache_append(cache, k, v, slots, ...)       the drafted tokens, as any others
    attend_tree(out, q, cache, table, lens)     each over its row and its own branch
    cache_compact(cache, table, picks, counts)  the accepted ones together
    cache_copy(cache, src, dst)                 pages to pages, where requests fork or move

Conventions as in ``decode.py``: the functions check and marshal, work is
enqueued on the caller's current stream of the cache's device (or ``stream``),
and nothing synchronizes.  A call goes to ``_bind`` first; what that leaves comes
back to the checks here.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import LIB_PATH, _check, _stream_handle as _stream, load as _load
from . import decode as _d

MAX_DRAFTS = 64

_p, _q, _i, _f = _d._p, _d._q, _d._i, _d._f


class TreeC(ctypes.Structure):
    _fields_ = [("attend", _d.AttendC), ("masks", _p), ("counts", _p), ("depths", _p), ("slopes", _p), ("q_draft", _q),
                ("out_draft", _q), ("cap", _f), ("drafts", _i)]


class CompactC(ctypes.Structure):
    _fields_ = [("table", _p), ("to", _p), ("picks", _p), ("counts", _p), ("starts", _p), ("batch", _q), ("most", _q),
                ("table_row", _q), ("table_width", _q), ("to_row", _q), ("to_width", _q)]


_TREE = struct.Struct("PPPPqqfi")  # what follows the attention's own arguments
_COMPACT = _d._packer(CompactC)


def bind(lib) -> None:
    """Argument types of the drafted step's entry points."""
    text, i64p = ctypes.c_char_p, ctypes.POINTER(_q)
    lib.detfold_attend_tree.argtypes = [text, text, _p]
    lib.detfold_plan_tree.argtypes = [text, _q, _i, _i, _q, _q, _i, _i, _i, _i, ctypes.POINTER(_d.AttendPlan)]
    lib.detfold_tree_workspace.argtypes = [text, _q, _i, _i, _q, _i, i64p]
    lib.detfold_cache_copy.argtypes = [text, text, _p, _p, _p, _q, _p]
    lib.detfold_cache_compact.argtypes = [text, text, _p]


_native = None


def _bound():
    """As ``decode._bound``: ``_bind``'s functions, each with the library's own, and torch's accessors of the
    current stream and device; where there is none of this library's build, functions that take no call."""
    global _native
    lib = _load()
    try:
        import torch
        from . import _bind
        with open(LIB_PATH + ".sha256") as f:
            ok = f.read().strip() == _bind.built_from
        raw, here = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    except (ImportError, OSError, AttributeError):
        ok = False
    if ok:
        _native = raw, here, *(x for call, of in ((_bind.tree, lib.detfold_attend_tree),
                                                  (_bind.copy, lib.detfold_cache_copy),
                                                  (_bind.compact, lib.detfold_cache_compact))
                               for x in (call, ctypes.cast(of, _p).value))
    else:
        _native = (lambda device: 0, lambda: 0, *(lambda *args: -1, 0) * 3)
    return _native


def _on_device(dev: int, f, *args) -> int:
    """The library's call with the cache's device current."""
    import torch
    if torch.cuda.current_device() == dev:
        return f(*args)
    with torch.cuda.device(dev):
        return f(*args)


def _workspace(cache, batch: int, drafts: int, q_heads: int, max_len: int, split: int) -> int:
    n = ctypes.c_int64()
    _check(_on_device(cache.device_index, _load().detfold_tree_workspace, cache._c, batch, drafts, q_heads, max_len, split,
                      ctypes.byref(n)), "attend_workspace")
    return n.value


def plan_tree(cache, batch: int, drafts: int, q_heads: int, max_len: int, cu_count: int, *, type: int = _d.BF16,
              out_type=None, window: int = 0, split: int = 0) -> dict:
    """How ``attend_tree`` would split such a call (host only): ``cache`` is a ``PagedCache`` or the bytes of a
    ``PagedCacheC``."""
    p = _d.AttendPlan()
    _check(_load().detfold_plan_tree(cache._c if isinstance(cache, _d.PagedCache) else bytes(cache), batch, drafts, q_heads,
                                     max_len, window, split, type, type if out_type is None else out_type, cu_count,
                                     ctypes.byref(p)), "plan_tree")
    return p.as_dict()


def attend_tree(out, q, cache, table, lens, *, masks=None, counts=None, depths=None, cap: float = 0.0, slopes=None, scale=None,
                window: int = 0, max_len=None, lse=None, workspace=None, split: int = 0, stream=None) -> None:
    """Attention of a tree of drafted tokens per row: ``out`` [batch, drafts, q_heads, v_dim] and, where given, ``lse``
    [batch, drafts, q_heads] (float32) of ``q`` [batch, drafts, q_heads, dim] over the first ``lens`` (int32) tokens
    of each row, of which the last ones are the drafted tokens themselves (``cache_append`` stored them), in q's
    order; at most 64.

    A drafted token sees the row's prefix, and drafted token j if bit j of its ``masks`` (int64 [batch, drafts]) is
    set, its own bit too; without masks the tokens are a chain.  ``counts`` (int32 [batch]): a row's number of drafted
    tokens where it is smaller; the outputs behind it stay as they were.  ``depths`` (int32 [batch, drafts], 0 to 63;
    default: a token's number) are their positions after the prefix, which ``window`` and ``slopes`` go by: both need
    them where there are masks.  With ``window`` a token sees less than so many positions back.

    ``cap`` > 0: scores become cap * tanh(score / cap); then ``slopes`` (float32 [q_heads]) add slope * (position of
    the token seen - own position); none of these, nor ``scale``, may pass 2^127.  A key scale that is no number, or
    takes ``scale`` past that, gives NaN.  A token that sees nothing gives 0 and -infinity.  All else as
    ``attend_paged``, the ``workspace`` from ``attend_workspace(..., drafts=drafts)``."""
    dev = cache.device_index
    raw, here, call, of = (_native or _bound())[:4]
    if here() == dev:
        rc = call(of, cache, dev, raw(dev) if stream is None else int(stream.cuda_stream), out, q, table, lens, masks, counts,
                  depths, cap, slopes, 1.0 / math.sqrt(cache.dim) if scale is None else scale, window, max_len, lse, workspace, split, 4)
        if rc >= 0:
            return _check(rc, "attend_tree") if rc else None
    if q.dim() != 4:
        raise ValueError("q must be [batch, drafts, q_heads, %d], got %s" % (cache.dim, tuple(q.shape)))
    _attend("attend_tree", out, q, cache, table, lens, masks, counts, depths, cap, slopes, scale, window, max_len, lse, workspace,
            split, stream)


def scored(out, q, cache, table, lens, cap, slopes, scale, window, max_len, lse, workspace, split, stream) -> None:
    """``attend_paged`` with capped or biased scores: a tree of one token."""
    dev = cache.device_index
    raw, here, call, of = (_native or _bound())[:4]
    if here() == dev:
        rc = call(of, cache, dev, raw(dev) if stream is None else int(stream.cuda_stream), out, q, table, lens, None, None,
                  None, cap, slopes, 1.0 / math.sqrt(cache.dim) if scale is None else scale, window, max_len, lse, workspace, split, 3)
        if rc >= 0:
            return _check(rc, "attend_paged") if rc else None
    for x, name in ((q, "q"), (out, "out")):
        if x.dim() != 3:
            raise ValueError("%s must be [batch, q_heads, dim], got %s" % (name, tuple(x.shape)))
    if lse is not None and lse.dim() != 2:
        raise ValueError("lse must be [batch, q_heads], got %s" % (tuple(lse.shape),))
    _attend("attend_paged", out[:, None], q[:, None], cache, table, lens, None, None, None, cap, slopes, scale, window, max_len,
            None if lse is None else lse[:, None], workspace, split, stream)


def _attend(what, out, q, cache, table, lens, masks, counts, depths, cap, slopes, scale, window, max_len, lse, workspace, split,
            stream) -> None:
    dev = cache.device_index
    type_, out_type = _d._type(q, "q"), _d._type(out, "out")
    if out_type != type_ and out_type != _d.F32:
        _d._refuse_type(out, "out", "of q's type or float32")
    batch, drafts, q_heads, dim = q.shape
    if dim != cache.dim:
        raise ValueError("q must have heads of %d, got %s" % (cache.dim, tuple(q.shape)))
    if tuple(out.shape) != (batch, drafts, q_heads, cache.v_dim):
        raise ValueError("out must have shape %s, got %s" % ((batch, drafts, q_heads, cache.v_dim), tuple(out.shape)))
    if not 1 <= drafts <= MAX_DRAFTS:
        raise ValueError("q must have 1 to %d drafted tokens, got %d" % (MAX_DRAFTS, drafts))
    qs, os = _d._place(q, "q", dev), _d._place(out, "out", dev)
    lens_p = _d._plain(lens, "lens", dev, "int32", (batch,))
    ts, width = _table(table, "table", dev, batch)
    masks_p, counts_p, depths_p, slopes_p, lse_p = (
        0 if t is None else _d._plain(t, name, dev, kind, shape)
        for t, name, kind, shape in ((masks, "masks", "int64", (batch, drafts)), (counts, "counts", "int32", (batch,)),
                                     (depths, "depths", "int32", (batch, drafts)), (slopes, "slopes", "float32", (q_heads,)),
                                     (lse, "lse", "float32", (batch, drafts, q_heads))))
    if cap and ctypes.c_float(cap).value == 0.0:  # in the library 0 is no cap at all
        raise ValueError("cap must be 0 or a normal float32, got %r" % (cap,))
    if masks is not None and depths is None and (window or slopes is not None):
        raise ValueError("masks with a window or slopes need depths")
    if max_len is None:
        max_len = min(width * cache.page, 2 ** 31 - 1 - MAX_DRAFTS)
    if workspace is None:  # in the pool of the stream that uses it, as attend_paged's
        import torch
        with _d._within(stream, dev):
            workspace = torch.empty(_workspace(cache, batch, drafts, q_heads, max_len, split), dtype=torch.uint8, device=cache.k.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    args = _d._ATTEND.pack(out.data_ptr(), q.data_ptr(), lse_p, table.data_ptr(), lens_p, workspace.data_ptr(), workspace.nbytes,
                           batch, max_len, window, ts[0], width, qs[0], qs[2], os[0], os[2],
                           1.0 / math.sqrt(cache.dim) if scale is None else scale, type_, out_type, q_heads, split, 0)
    args += _TREE.pack(masks_p, counts_p, depths_p, slopes_p, qs[1], os[1], cap, drafts)
    _check(_on_device(dev, _load().detfold_attend_tree, cache._described(), args, _stream(q, stream)), what)


def _table(t, name: str, dev: int, batch: int):
    """The strides of a table of pages, int32 [batch, width], and its width."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != torch.int32:
        _d._refuse_type(t, name, "int32")
    if t.dim() != 2 or t.shape[0] != batch:
        raise ValueError("%s must be [%d, width], got %s" % (name, batch, tuple(t.shape)))
    return _d._place(t, name, dev), t.shape[1]


def cache_copy(cache, src, dst, *, tokens=None, into=None, stream=None) -> None:
    """Copy pages: page ``dst[i]`` becomes what page ``src[i]`` holds, keys and values (int32 [count] each).  With
    ``tokens`` (int32 [count]) only the first ``tokens[i]`` slots of a page; with ``into``, another ``PagedCache`` of
    the same page size, heads, head sizes and type, the pages of that one are written; one whose values are a view of
    its keys takes copies of such caches alone.

    A pair of which either page is not in its cache (-1) is left out.  The copies run in no order: no page may be both
    written and read, or written twice, in one call.  Scales are not copied."""
    dev = cache.device_index
    raw, here, _, _, call, of = (_native or _bound())[:6]
    if here() == dev:
        rc = call(of, cache, dev, raw(dev) if stream is None else int(stream.cuda_stream), src, dst, tokens, into)
        if rc >= 0:
            return _check(rc, "cache_copy") if rc else None
    count = src.shape[0] if getattr(src, "ndim", 0) == 1 else -1
    if count < 0:
        raise ValueError("src must be an int32 tensor [count]")
    src_p, dst_p, tokens_p = (0 if t is None else _d._plain(t, name, dev, "int32", (count,))
                              for t, name in ((src, "src"), (dst, "dst"), (tokens, "tokens")))
    if dst is None:
        raise TypeError("dst must be a torch.Tensor")
    if into is not None and (into.device_index, into.type, into.page, into.heads, into.dim, into.v_dim) != (
            dev, cache.type, cache.page, cache.heads, cache.dim, cache.v_dim):
        raise ValueError("into must be a cache of the same device, type, page size, heads and head sizes")
    _check(_on_device(dev, _load().detfold_cache_copy, cache._described(), None if into is None else into._described(),
                      src_p, dst_p, tokens_p, count, _stream(src, stream)), "cache_copy")


def cache_compact(cache, table, picks, counts, *, starts=None, to=None, stream=None) -> None:
    """Move each row's kept tokens together: for i below ``counts[b]`` (int32 [batch]) token ``starts[b] + i`` of row b
    becomes what token ``starts[b] + picks[b, i]`` was (int32 [batch, most]; ``starts``: int32 [batch], default 0).
    ``table`` (int32 [batch, width]) names the rows' pages.

    In place, as if all tokens were read before any is written; a pick below its own i is left out.  A cache whose
    values are a view within its keys, or its keys within its values, or whose heads are one (expanded), moves once;
    one whose tokens share memory otherwise is refused.  With ``to`` (int32 [batch, width]) the tokens go to the pages
    that it names, of which none may be read in this call.  Moves from or to tokens that the tables, or the cache, do
    not have are left out.  A written page may be one row's only."""
    dev = cache.device_index
    native = _native or _bound()
    raw, here, call, of = native[0], native[1], native[6], native[7]
    if here() == dev:
        rc = call(of, cache, dev, raw(dev) if stream is None else int(stream.cuda_stream), table, picks, counts, starts, to)
        if rc >= 0:
            return _check(rc, "cache_compact") if rc else None
    if getattr(picks, "ndim", 0) != 2:
        raise ValueError("picks must be an int32 tensor [batch, most]")
    batch, most = picks.shape
    picks_p = _d._plain(picks, "picks", dev, "int32", (batch, most))
    counts_p = _d._plain(counts, "counts", dev, "int32", (batch,))
    starts_p = 0 if starts is None else _d._plain(starts, "starts", dev, "int32", (batch,))
    ts, width = _table(table, "table", dev, batch)
    to_p = to_row = to_width = 0
    if to is not None:
        os, to_width = _table(to, "to", dev, batch)
        to_row = os[0]
        to_p = to.data_ptr()
        if not to_p:  # no page to move to
            return
    args = _COMPACT.pack(table.data_ptr(), to_p, picks_p, counts_p, starts_p, batch, most, ts[0], width, to_row, to_width)
    _check(_on_device(dev, _load().detfold_cache_compact, cache._described(), args, _stream(picks, stream)), "cache_compact")
