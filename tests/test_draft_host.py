"""Host-side checks of the drafted step's C ABI (CPU only).  Every call fails
validation or has nothing to do, so no address is ever handed to a kernel."""
import ctypes
import math
import re

import pytest

import test_abi_host
from deterministic_fixed_order_amd import decode as d
from deterministic_fixed_order_amd import draft
from test_decode_host import (BAD_CACHES, BF, E4, F16, F32, K, LENS, LSE, OUT, Q, TABLE, V, WORK, cache)

SIDE = 0x7F8000000000


def attend(**kw):
    a = d.AttendC(out=OUT, q=Q, lse=LSE, table=TABLE, lens=LENS, workspace=WORK, workspace_bytes=1 << 30, batch=3,
                  max_len=640, table_row=40, table_width=40, q_row=5 * 256, q_head=64, out_row=5 * 128, out_head=32,
                  scale=0.125, type=BF, out_type=BF, q_heads=4)
    t = draft.TreeC(attend=a, masks=SIDE, counts=SIDE + 4096, depths=SIDE + 8192, slopes=SIDE + 12288, q_draft=256, out_draft=128,
                    cap=30.0, drafts=5)
    for k, v in kw.items():
        setattr(t if k in dict(t._fields_) else t.attend, k, v)
    return bytes(t)


def compact(**kw):
    a = draft.CompactC(table=TABLE, to=TABLE + 4096, picks=SIDE, counts=SIDE + 4096, starts=SIDE + 8192, batch=3, most=7, table_row=40,
                       table_width=40, to_row=9, to_width=9)
    for k, v in kw.items():
        setattr(a, k, v)
    return bytes(a)


@pytest.fixture(scope="module")
def lib(detfold_lib):
    return detfold_lib.load()


def test_structs_are_laid_out_as_the_header_has_them():
    text = re.sub(r"/\*.*?\*/", "", open(test_abi_host.HEADER).read(), flags=re.S)
    ctype = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float, "detfold_attend": d.AttendC}
    for name, struct in (("detfold_tree", draft.TreeC), ("detfold_compact", draft.CompactC)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        fields = []
        for line in filter(None, (x.strip() for x in body.split(";"))):
            kind, names = re.match(r"(?:const\s+)?(\w+)\s+(.*)$", line, re.S).groups()
            for n in (x.strip() for x in names.split(",")):
                fields.append((n.lstrip("*"), ctypes.c_void_p if n.startswith("*") else ctype[kind]))
        assert fields == struct._fields_, name
    assert d._ATTEND.size + draft._TREE.size == ctypes.sizeof(draft.TreeC) and draft.TreeC.masks.offset == d._ATTEND.size
    assert draft._COMPACT.size == ctypes.sizeof(draft.CompactC)


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(lib, bad):
    c = cache(**bad)
    assert lib.detfold_attend_tree(c, attend(), None) == 1
    assert lib.detfold_plan_tree(c, 3, 5, 4, 640, 0, 0, BF, BF, 256, ctypes.byref(d.AttendPlan())) == 1
    assert lib.detfold_tree_workspace(c, 3, 5, 4, 640, 0, ctypes.byref(ctypes.c_int64())) == 1
    assert lib.detfold_cache_copy(c, None, SIDE, SIDE + 64, None, 3, None) == 1
    assert lib.detfold_cache_copy(cache(), c, SIDE, SIDE + 64, None, 3, None) == 1
    assert lib.detfold_cache_compact(c, compact(), None) == 1


@pytest.mark.parametrize("bad", [
    dict(out=0), dict(q=0), dict(lens=0), dict(table=0), dict(batch=-1), dict(batch=1 << 31), dict(max_len=-1),
    dict(max_len=1 << 31), dict(window=-1), dict(table_row=-1), dict(table_width=-1), dict(q_heads=0), dict(q_heads=3),
    dict(split=-32), dict(split=33), dict(type=F16), dict(type=E4), dict(out_type=F16), dict(scale=math.inf), dict(scale=math.nan),
    dict(q=Q + 1), dict(out=OUT + 1), dict(lse=LSE + 2), dict(table=TABLE + 2), dict(lens=LENS + 1), dict(workspace=WORK + 8),
    dict(workspace_bytes=-1), dict(q_row=-1), dict(q_draft=-1), dict(out_draft=-128), dict(out_row=1 << 60), dict(q_draft=1 << 60),
    dict(drafts=0), dict(drafts=-1), dict(drafts=65), dict(cap=-1.0), dict(cap=math.inf), dict(cap=math.nan), dict(masks=SIDE + 4),
    dict(counts=SIDE + 4098), dict(depths=SIDE + 8193), dict(slopes=SIDE + 12290), dict(depths=0), dict(depths=0, slopes=0, window=5),
    dict(reserved=1)], ids=str)
def test_bad_trees(lib, bad):
    assert lib.detfold_attend_tree(cache(), attend(**bad), None) == 1


def test_largest_scales(lib):
    """Scores are held times log2 e, and so are the cap and the scale: finite up to 2^127, which is no bad argument."""
    past = 2.0 ** 127 * (1 + 2.0 ** -23)
    for name in ("scale", "cap"):
        assert lib.detfold_attend_tree(cache(), attend(**{name: past}), None) == 1
        assert lib.detfold_attend_tree(cache(), attend(batch=0, **{name: 2.0 ** 127}), None) == 0
    assert lib.detfold_attend_tree(cache(), attend(scale=-past), None) == 1


@pytest.mark.parametrize("bad", [
    dict(out_head=31), dict(out_head=0), dict(out_draft=127), dict(out_draft=0), dict(out_row=639), dict(out_row=0), dict(out=Q),
    dict(out=K + 64), dict(out=V), dict(out=TABLE), dict(out=LENS), dict(out=LSE), dict(out=WORK + 16), dict(out=SIDE), dict(lse=Q),
    dict(lse=WORK), dict(lse=K), dict(lse=SIDE + 8192), dict(workspace=K), dict(workspace=Q - 64), dict(workspace=SIDE - 64),
    dict(out_head=128, out_draft=32, out_row=480)], ids=str)
def test_overlapping_trees(lib, bad):
    assert lib.detfold_attend_tree(cache(), attend(**bad), None) == 2


def test_types_that_go_together(lib):
    for t in (F32, BF, F16, E4):
        for ct in (F32, BF, F16, E4):
            ok = t != E4 and (ct == t or ct == E4 or (t == F32 and ct == BF))
            got = lib.detfold_attend_tree(cache(type=ct), attend(type=t, out_type=F32, batch=0), None)
            assert got == (0 if ok else 1), (t, ct)


def test_nothing_to_do(lib):
    nothing = dict(out=0, q=0, lse=0, table=0, lens=0, workspace=0, masks=0, counts=0, depths=0, slopes=0, batch=0)
    assert lib.detfold_attend_tree(cache(), attend(**nothing), None) == 0
    assert lib.detfold_cache_copy(cache(), None, None, None, None, 0, None) == 0
    for none in (dict(batch=0), dict(most=0)):
        assert lib.detfold_cache_compact(cache(), compact(table=0, to=0, picks=0, counts=0, starts=0, **none), None) == 0
    assert lib.detfold_attend_tree(None, attend(), None) == 1
    assert lib.detfold_attend_tree(cache(), None, None) == 1
    assert lib.detfold_cache_copy(None, None, SIDE, SIDE, None, 3, None) == 1
    assert lib.detfold_cache_compact(cache(), None, None) == 1
    assert lib.detfold_cache_compact(None, compact(), None) == 1


def test_copy_refusals(lib):
    def call(src=SIDE, dst=SIDE + 64, tokens=None, count=3, into=None, **kw):
        return lib.detfold_cache_copy(cache(**kw), into, src, dst, tokens, count, None)

    for bad in (dict(src=None), dict(dst=None), dict(src=SIDE + 2), dict(dst=SIDE + 1), dict(tokens=SIDE + 3), dict(count=-1),
                dict(count=1 << 31), dict(into=cache(page=8, k=Q, v=OUT)), dict(into=cache(heads=1, k=Q, v=OUT)),
                dict(into=cache(dim=60, k=Q, v=OUT)), dict(into=cache(v_dim=16, k=Q, v=OUT)), dict(into=cache(type=F16, k=Q, v=OUT)),
                dict(pages=1, page=(1 << 31) - 1, k_page=0, v_page=0)):
        assert call(**bad) == 1, bad
    for bad in (dict(src=K + 4), dict(dst=V + 8), dict(tokens=K), dict(into=cache(k=K + 2 * 64)), dict(into=cache(v=Q)),
                dict(into=cache(k=Q, v=OUT, k_head=128, k_token=256), src=Q + 64), dict(into=cache(k_head=1024, k_token=64))):
        assert call(**bad) == 2, bad


def test_compact_refusals(lib):
    for bad in (dict(batch=-1), dict(batch=1 << 31), dict(most=-1), dict(most=1 << 31), dict(table=0), dict(picks=0), dict(counts=0),
                dict(table=TABLE + 1), dict(to=TABLE + 2), dict(picks=SIDE + 1), dict(counts=SIDE + 2), dict(starts=SIDE + 3),
                dict(table_row=-1), dict(table_width=-1), dict(to_row=-1), dict(to_width=-1), dict(table_row=1 << 60)):
        assert lib.detfold_cache_compact(cache(), compact(**bad), None) == 1, bad
    for bad in (dict(table=K), dict(to=V + 64), dict(picks=K + 4), dict(counts=V), dict(starts=K)):
        assert lib.detfold_cache_compact(cache(), compact(**bad), None) == 2, bad


def _plan(lib, batch, drafts, q_heads, max_len, window=0, split=0, type=BF, out=None, cu=256, **kw):
    p = d.AttendPlan()
    assert lib.detfold_plan_tree(cache(**kw), batch, drafts, q_heads, max_len, window, split, type, type if out is None else out, cu,
                                 ctypes.byref(p)) == 0
    return p


def test_plan_covers_every_length(lib):
    for batch in (0, 1, 3, 64, 5000):
        for drafts in (1, 2, 8, 33, 64):
            for max_len in (0, 1, 31, 32, 33, 1000, 8192, 131072, (1 << 31) - 65):
                for window in (0, 1, 100, 1500):
                    for split in (0, 32, 4096):
                        if split and batch * max_len > 1 << 36:
                            continue  # more parts than a workspace is made for
                        for cu in (1, 64, 256):
                            p = _plan(lib, batch, drafts, 8, max_len, window, split, cu=cu)
                            seen = min(max_len, window + drafts - 1) if window else max_len
                            assert p.splits >= 1 and p.splits * p.split >= seen
                            assert p.splits == 1 or (p.splits - 1) * p.split < seen
                            if split:
                                assert p.split == split or p.splits == 1
                            assert (p.workspace_bytes > 0) == (p.splits > 1 and batch > 0)


@pytest.mark.parametrize("heads,group,dim", [(2, 4, 64), (8, 4, 128), (1, 1, 256), (3, 5, 84), (1, 24, 16), (16, 8, 128), (4, 40, 250)])
def test_workspace_serves_smaller_calls(lib, heads, group, dim):
    """A workspace of some sizes serves every smaller batch, length and number of drafted tokens, every window, every
    type of query, and the plain attention of one token."""
    import random
    rng = random.Random(heads * dim)
    kw = dict(heads=heads, dim=dim, v_dim=dim, k_head=dim, k_token=heads * dim, k_page=16 * heads * dim, v_head=dim,
              v_token=heads * dim, v_page=16 * heads * dim)
    for _ in range(60):
        batch, drafts = rng.choice([1, rng.randint(1, 300), 6000]), rng.randint(1, 64)
        max_len, split = rng.choice([rng.randint(1, 3000), rng.randint(1, 200000)]), rng.choice([0, 0, 64, 2048])
        if split and batch * heads * group * drafts * max_len // split > 1 << 38:
            continue
        most = _plan(lib, batch, drafts, heads * group, max_len, 0, split, F32, **kw).workspace_upto
        for _ in range(30):
            b, n, t = rng.randint(0, batch), rng.choice([max_len, rng.randint(0, max_len), rng.randint(0, 400)]), rng.randint(1, drafts)
            n, w = min(n, max_len), rng.choice([0, rng.randint(1, 5000)])
            type, out = rng.choice([(BF, BF), (BF, F32), (F32, F32)])
            p = _plan(lib, b, t, heads * group, n, w, split, type, out, **kw)
            assert p.workspace_bytes <= p.workspace_upto <= most, (batch, drafts, max_len, split, b, t, n, w)
            one = _plan(lib, b, 1, heads * group, n, w, split, type, out, **kw)
            plain = d.AttendPlan()
            assert lib.detfold_plan_attend(cache(**kw), batch, heads * group, max_len, 0, split, 256, ctypes.byref(plain)) == 0
            assert one.workspace_bytes <= plain.workspace_upto, (batch, max_len, split, b, n, w)


def test_plan_refusals(lib):
    ok = dict(batch=3, drafts=5, q_heads=4, max_len=640, window=0, split=0, type=BF, out=BF, cu=256)
    for bad in (dict(drafts=0), dict(drafts=65), dict(q_heads=3), dict(max_len=(1 << 31) - 64), dict(type=F16), dict(out=F16), dict(type=E4),
                dict(cu=0), dict(split=31), dict(window=-1), dict(batch=-1)):
        a = {**ok, **bad}
        assert lib.detfold_plan_tree(cache(), a["batch"], a["drafts"], a["q_heads"], a["max_len"], a["window"], a["split"], a["type"],
                                     a["out"], a["cu"], ctypes.byref(d.AttendPlan())) == 1, bad
    assert lib.detfold_plan_tree(cache(), 3, 5, 4, 640, 0, 0, BF, BF, 256, None) == 1
    assert lib.detfold_tree_workspace(cache(), 3, 5, 4, 640, 0, None) == 1
