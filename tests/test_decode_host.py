"""Host-side checks of the decode-step operators' C ABI (CPU only).  Every call
fails validation or has nothing to do, so no address is ever handed to a
kernel: bad arguments are refused before the device is touched."""
import ctypes
import math
import re

import pytest

import test_abi_host
from deterministic_fixed_order_amd import decode as d

K, V, Q, OUT, LSE, TABLE, LENS, WORK = (0x7F0000000000 + (i << 36) for i in range(8))
BF, F32, F16, E4 = d.BF16, d.F32, d.F16, d.E4M3


def _bytes(struct):
    return bytes(struct)


def cache(**kw):
    c = d.PagedCacheC(k=K, v=V, pages=100, k_page=16 * 2 * 64, k_token=2 * 64, k_head=64, v_page=16 * 2 * 32,
                      v_token=2 * 32, v_head=32, page=16, heads=2, dim=64, v_dim=32, type=BF)
    for k, v in kw.items():
        setattr(c, k, v)
    return _bytes(c)


def append(**kw):
    a = d.AppendC(k=Q, v=Q + (1 << 30), q=Q + (1 << 31), q_out=OUT, slots=LENS, positions=LENS + 4096, cos=TABLE,
                  sin=TABLE + (1 << 30), tokens=5, angles=1000, k_token=128, k_head=64, v_token=64, v_head=32,
                  q_token=256, q_head=64, out_token=256, out_head=64, type=BF, q_heads=4, rot=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return _bytes(a)


def attend(**kw):
    a = d.AttendC(out=OUT, q=Q, lse=LSE, table=TABLE, lens=LENS, workspace=WORK, workspace_bytes=1 << 30, batch=3,
                  max_len=640, table_row=40, table_width=40, q_row=256, q_head=64, out_row=128, out_head=32,
                  scale=0.125, type=BF, out_type=BF, q_heads=4)
    for k, v in kw.items():
        setattr(a, k, v)
    return _bytes(a)


@pytest.fixture(scope="module")
def lib(detfold_lib):
    return detfold_lib.load()


def test_structs_are_laid_out_as_the_header_has_them():
    text = re.sub(r"/\*.*?\*/", "", open(test_abi_host.HEADER).read(), flags=re.S)
    ctype = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float}
    for name, struct in (("detfold_paged_cache", d.PagedCacheC), ("detfold_append", d.AppendC),
                         ("detfold_attend", d.AttendC), ("detfold_attend_plan", d.AttendPlan)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        fields = []
        for line in body.split(";"):
            line = line.strip()
            if not line:
                continue
            kind, names = re.match(r"(?:const\s+)?(\w+)\s+(.*)$", line, re.S).groups()
            for n in names.split(","):
                n = n.strip()
                fields.append((n.lstrip("*"), ctypes.c_void_p if n.startswith("*") else ctype[kind]))
        assert fields == struct._fields_, name
    for packer, struct in ((d._CACHE, d.PagedCacheC), (d._APPEND, d.AppendC), (d._ATTEND, d.AttendC)):
        assert packer.size == ctypes.sizeof(struct)


BAD_CACHES = [dict(k=0), dict(v=0), dict(k=K + 1), dict(v=V + 1), dict(type=4), dict(type=-1), dict(pages=0),
              dict(page=0), dict(page=-3), dict(pages=1 << 40), dict(pages=1 << 28, page=16), dict(heads=0),
              dict(heads=1 << 20), dict(dim=15), dict(dim=257), dict(v_dim=8), dict(v_dim=300), dict(k_page=-1),
              dict(k_token=-64), dict(v_head=-1), dict(k_page=1 << 60), dict(v_page=1 << 45), dict(k_scale=TABLE),
              dict(type=E4, k_scale=TABLE + 2), dict(type=E4, v_scale=TABLE + 1), dict(reserved=1)]


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(lib, bad):
    c = cache(**bad)
    assert lib.detfold_cache_append(c, append(), None) == 1
    assert lib.detfold_attend_paged(c, attend(), None) == 1
    assert lib.detfold_plan_attend(c, 3, 4, 640, 0, 0, 256, ctypes.byref(d.AttendPlan())) == 1
    assert lib.detfold_attend_workspace(c, 3, 4, 640, 0, ctypes.byref(ctypes.c_int64())) == 1


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(tokens=1 << 31), dict(k=0), dict(v=0), dict(q=0), dict(q_out=0), dict(slots=0), dict(q_heads=0),
    dict(q_heads=-1), dict(rot=-2), dict(rot=63), dict(rot=66), dict(pairs=2), dict(pairs=-1), dict(angles=0), dict(angles=-1),
    dict(positions=0), dict(cos=0), dict(sin=0), dict(type=E4), dict(type=F32, k=Q + 2), dict(type=F16), dict(type=7),
    dict(k=Q + 1), dict(q=Q + (1 << 31) + 1), dict(q_out=OUT + 1), dict(slots=LENS + 4), dict(positions=LENS + 4100),
    dict(cos=TABLE + 2), dict(k_token=-1), dict(v_head=-1), dict(q_token=1 << 60), dict(out_head=-64)], ids=str)
def test_bad_appends(lib, bad):
    assert lib.detfold_cache_append(cache(), append(**bad), None) == 1


@pytest.mark.parametrize("bad", [
    dict(out_head=63), dict(out_head=0), dict(out_token=255), dict(out_token=0),  # heads of q_out meet
    dict(q_out=Q + (1 << 31)), dict(q_out=Q + (1 << 31), out_token=512, q_token=512, out_head=64, q_head=128),
    dict(q_out=K + 4096), dict(k=K), dict(v=V + 100 * 1024 * 2 - 2), dict(q=K + 64), dict(slots=K + 8), dict(cos=V + 4),
    dict(positions=OUT + 8), dict(q_out=LENS), dict(q_out=Q), dict(k=OUT)], ids=str)
def test_overlapping_appends(lib, bad):
    if bad == dict(q_out=Q + (1 << 31)):  # q itself: in place
        a = append(tokens=0, **bad)
        assert lib.detfold_cache_append(cache(), a, None) == 0
        return
    assert lib.detfold_cache_append(cache(), append(**bad), None) == 2


@pytest.mark.parametrize("bad", [
    dict(out=0), dict(q=0), dict(lens=0), dict(table=0), dict(batch=-1), dict(batch=1 << 31), dict(max_len=-1),
    dict(max_len=1 << 31), dict(window=-1), dict(table_row=-1), dict(table_width=-1), dict(q_heads=0), dict(q_heads=3),
    dict(q_heads=-2), dict(split=-32), dict(split=33), dict(split=1), dict(type=F16), dict(type=E4), dict(type=9),
    dict(out_type=F16), dict(out_type=E4), dict(scale=math.inf), dict(scale=math.nan), dict(q=Q + 1), dict(out=OUT + 1),
    dict(lse=LSE + 2), dict(table=TABLE + 2), dict(lens=LENS + 1), dict(workspace=WORK + 8), dict(workspace_bytes=-1),
    dict(q_row=-1), dict(q_head=-1), dict(out_row=-1), dict(out_row=1 << 60), dict(table_row=1 << 60),
    dict(reserved=1)], ids=str)
def test_bad_attends(lib, bad):
    assert lib.detfold_attend_paged(cache(), attend(**bad), None) == 1


@pytest.mark.parametrize("bad", [
    dict(out_head=31), dict(out_head=0), dict(out_row=127), dict(out_row=0), dict(out=Q), dict(out=K + 64), dict(out=V),
    dict(out=TABLE), dict(out=LENS), dict(out=LSE), dict(out=WORK + 16), dict(lse=Q), dict(lse=WORK), dict(lse=K),
    dict(workspace=K), dict(workspace=Q - 64)], ids=str)
def test_overlapping_attends(lib, bad):
    assert lib.detfold_attend_paged(cache(), attend(**bad), None) == 2


def test_types_that_go_together(lib):
    for t in (F32, BF, F16, E4):
        for ct in (F32, BF, F16, E4):
            ok = t != E4 and (ct == t or ct == E4 or (t == F32 and ct == BF))
            got = lib.detfold_cache_append(cache(type=ct), append(type=t, tokens=0), None)
            assert got == (0 if ok else 1), (t, ct)
            got = lib.detfold_attend_paged(cache(type=ct), attend(type=t, out_type=F32, batch=0), None)
            assert got == (0 if ok else 1), (t, ct)


def test_nothing_to_do(lib):
    empty = dict(k=0, v=0, q=0, q_out=0, slots=0, positions=0, cos=0, sin=0, tokens=0)
    assert lib.detfold_cache_append(cache(), append(**empty), None) == 0
    assert lib.detfold_attend_paged(cache(), attend(out=0, q=0, lse=0, table=0, lens=0, workspace=0, batch=0), None) == 0
    assert lib.detfold_fold_softmax(None, None, None, None, F32, 2, 0, 8, 0, 0, None) == 0
    assert lib.detfold_cache_append(None, append(), None) == 1
    assert lib.detfold_cache_append(cache(), None, None) == 1
    assert lib.detfold_attend_paged(None, attend(), None) == 1
    assert lib.detfold_attend_paged(cache(), None, None) == 1


def test_fold_softmax_refusals(lib):
    f = lib.detfold_fold_softmax
    ok = dict(out=OUT, outs=Q, lses=TABLE, lse=LSE, type=F32, W=3, rows=10, dim=8, op=80, lp=10)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["out"], a["outs"], a["lses"], a["lse"], a["type"], a["W"], a["rows"], a["dim"], a["op"], a["lp"], None)

    for bad in (dict(W=0), dict(W=-1), dict(rows=-1), dict(dim=0), dict(dim=-4), dict(type=E4), dict(type=-1), dict(out=None),
                dict(outs=None), dict(lses=None), dict(op=79), dict(lp=9), dict(op=1 << 62), dict(rows=1 << 62), dict(out=OUT + 2),
                dict(outs=Q + 1), dict(lses=TABLE + 2), dict(lse=LSE + 1)):
        assert call(**bad) == 1, bad
    for bad in (dict(out=Q), dict(out=Q + 80 * 4 * 3 - 4), dict(lse=TABLE), dict(lse=Q + 4), dict(out=TABLE + 8), dict(lse=OUT)):
        assert call(**bad) == 2, bad


def _plan(lib, batch, q_heads, max_len, window=0, split=0, cu=256, **kw):
    p = d.AttendPlan()
    assert lib.detfold_plan_attend(cache(**kw), batch, q_heads, max_len, window, split, cu, ctypes.byref(p)) == 0
    return p


def test_plan_covers_every_length(lib):
    for batch in (0, 1, 3, 64, 256, 5000):
        for max_len in (0, 1, 31, 32, 33, 1000, 8192, 131072, (1 << 31) - 1):
            for window in (0, 1, 100, 1500):
                for split in (0, 32, 4096):
                    for cu in (1, 64, 256):
                        p = _plan(lib, batch, 8, max_len, window, split, cu)
                        seen = min(max_len, window) if window else max_len
                        assert p.splits >= 1 and p.splits * p.split >= seen
                        assert p.splits == 1 or (p.splits - 1) * p.split < seen
                        if split:
                            assert p.split == split or p.splits == 1
                        assert (p.workspace_bytes > 0) == (p.splits > 1 and batch > 0)


def test_workspace_serves_smaller_calls(lib):
    """A workspace of some sizes serves every smaller batch, length and window."""
    import random
    rng = random.Random(3)
    for _ in range(300):
        batch, max_len, split = rng.randint(1, 300), rng.randint(1, 200000), rng.choice([0, 0, 64, 2048])
        most = _plan(lib, batch, 8, max_len, 0, split).workspace_upto
        for _ in range(20):
            b, n = rng.randint(0, batch), rng.randint(0, max_len)
            w = rng.choice([0, rng.randint(1, 5000)])
            p = _plan(lib, b, 8, n, w, split)
            assert p.workspace_bytes <= p.workspace_upto <= most, (batch, max_len, split, b, n, w)


def test_divider_is_exact():
    """The page division of the kernels: multiply and shift, for every divisor."""
    import random
    rng = random.Random(4)
    for dv in list(range(1, 300)) + [2 ** k + e for k in range(9, 31) for e in (-1, 0, 1)] + [2 ** 31 - 1]:
        s = (dv - 1).bit_length()
        m = -(-(1 << (31 + s)) // dv)
        assert m < 1 << 32
        xs = [0, 1, dv - 1, dv, dv + 1, 2 ** 31 - 1, 2 ** 31 - 2] + [rng.randrange(1 << 31) for _ in range(50)]
        for x in xs + [x // dv * dv for x in xs] + [x // dv * dv - 1 for x in xs if x >= dv]:
            if 0 <= x < 1 << 31:
                assert (x * m) >> (31 + s) == x // dv
