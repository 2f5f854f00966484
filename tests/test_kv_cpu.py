"""The key-value cache's calls refuse bad arguments before anything is launched: the C entry points by status,
the binding by ValueError.  CPU only, no pointer is followed."""
import ctypes as C

import numpy as np
import pytest

import moe_expert_amd as M
from tests import kv_refs as R
from tests.test_operators_cpu import Fake, refused

FAKE = C.c_void_p(0x100000)
ODD = C.c_void_p(0x100001)
TWO = C.c_void_p(0x100002)
EIGHT = C.c_void_p(0x100008)


def struct(**kw):
    a = dict(ktype=M.QMM_F16, vtype=M.QMM_Q8_0, k=0x100000, v=0x200000, kstride=4 * 64 * 256, vstride=4 * 64 * 136, npages=9, page_size=64,
             nheads=4, head_dim=128)
    a.update(kw)
    return M._KvStruct(*a.values())


ROWS = dict(cache=None, pages=FAKE, ldpages=5, max_pages=5, lens=FAKE, seg_off=FAKE, nseq=3, xtype=1, k=FAKE, ldk=512, v=FAKE, ldv=512, ntok=7,
            stream=None)
ATTEND = dict(cache=None, pages=FAKE, ldpages=5, max_pages=5, lens=FAKE, seg_off=FAKE, nseq=3, qtype=1, q=FAKE, ldq=1024, ntok=7, nheads=8,
              scale=0.1, window=0, otype=1, out=FAKE, ldo=1024, lse=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)


def call(fn, defaults, kw):
    """The call with kw's arguments and, for names that are no argument, fields of the cache."""
    a = dict(defaults)
    cache = struct(**{n: v for n, v in kw.items() if n not in defaults})
    a.update({n: v for n, v in kw.items() if n in defaults})
    a["cache"] = None if kw.get("cache", 1) is None else C.addressof(cache)
    return getattr(M.lib(), fn)(*a.values())


#: what every call says of the cache and the sequences (k and v of the cache are in `of_cache`)
SHARED = [
    (dict(cache=None), -1), (dict(ktype=9), -1), (dict(vtype=M.QMM_CB3), -1), (dict(npages=0), -1), (dict(page_size=0), -1), (dict(nheads=0), -1),
    (dict(page_size=40), -2), (dict(page_size=8192, kstride=1 << 30, vstride=1 << 30), -2), (dict(head_dim=32), -2), (dict(head_dim=160), -2),
    (dict(npages=1 << 31), -2), (dict(kstride=4 * 64 * 256 - 16), -1), (dict(vstride=4 * 64 * 136 - 16), -1), (dict(kstride=4 * 64 * 256 + 8), -3),
    (dict(vstride=4 * 64 * 136 + 2), -3), (dict(pages=None), -1), (dict(lens=None), -1), (dict(max_pages=0), -1), (dict(ldpages=4), -1),
    (dict(nseq=-1), -1), (dict(ntok=-1), -1), (dict(seg_off=None), -1), (dict(nseq=(1 << 14) + 1), -2), (dict(ntok=(1 << 20) + 1), -2),
    (dict(max_pages=(1 << 24) + 1, ldpages=1 << 25), -2), (dict(max_pages=1 << 40, ldpages=1 << 40), -2), (dict(pages=TWO), -3), (dict(lens=TWO), -3), (dict(seg_off=TWO), -3), (dict(ntok=0), 0),
    (dict(nseq=0, pages=None, lens=None), 0),
]


@pytest.mark.parametrize("kw,expect", SHARED)
@pytest.mark.parametrize("fn", ["qmm_kv_write", "qmm_kv_read", "qmm_kv_attend"])
def test_cache_and_sequences(fn, kw, expect):
    if fn == "qmm_kv_attend" and "nheads" in kw:
        return  # there it is the queries' number, tested below
    assert call(fn, ATTEND if fn == "qmm_kv_attend" else ROWS, kw) == expect


def of_cache(fn, defaults, **kw):
    a = dict(defaults)
    cache = struct(**kw)
    a["cache"] = C.addressof(cache)
    return getattr(M.lib(), fn)(*a.values())


@pytest.mark.parametrize("fn,defaults", [("qmm_kv_write", ROWS), ("qmm_kv_read", ROWS), ("qmm_kv_attend", ATTEND)])
def test_cache_pointers(fn, defaults):
    assert of_cache(fn, defaults, k=None) == -1 and of_cache(fn, defaults, v=None) == -1
    assert of_cache(fn, defaults, k=0x100008) == -3 and of_cache(fn, defaults, v=0x100004) == -3
    assert of_cache(fn, defaults, nheads=1025, kstride=1 << 30, vstride=1 << 30) == -2


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None, v=None), -1), (dict(xtype=0), -1), (dict(xtype=4), -1), (dict(ldk=511), -1), (dict(ldv=511), -1), (dict(k=TWO), -3),
    (dict(v=TWO), -3), (dict(k=ODD, xtype=2), -3), (dict(ntok=0, k=None, v=None), 0),
])
@pytest.mark.parametrize("fn", ["qmm_kv_write", "qmm_kv_read"])
def test_rows(fn, kw, expect):
    a = dict(ROWS)
    a.update(kw)
    cache = struct()
    a["cache"] = C.addressof(cache)
    assert getattr(M.lib(), fn)(*a.values()) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(qtype=0), -1), (dict(otype=7), -1), (dict(ldq=1023), -1), (dict(ldo=1023), -1),
    (dict(nheads=6), -1), (dict(nheads=0), -1), (dict(nheads=1028, ldq=1 << 20, ldo=1 << 20), -2), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(window=-1), -1), (dict(q=TWO), -3), (dict(out=TWO), -3), (dict(lse=TWO), -3), (dict(ws=EIGHT), -3),
    (dict(ws_bytes=0), -5), (dict(ntok=1 << 20, nheads=256, ldq=1 << 15, ldo=1 << 15), -2), (dict(ntok=0, q=None, out=None, ws=None), 0),
])
def test_attend(kw, expect):
    a = dict(ATTEND)
    a.update(kw)
    cache = struct()
    a["cache"] = C.addressof(cache)
    assert M.lib().qmm_kv_attend(*a.values()) == expect


@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 128), (4, 256), (8, 96)])
def test_workspace_is_enough_for_smaller_calls(heads, dim):
    cache = struct(nheads=heads, head_dim=dim, kstride=1 << 30, vstride=1 << 30)
    need = np.array([[[[M.lib().qmm_kv_attend_workspace(C.addressof(cache), n, heads * g, s, p) for p in (1, 2, 5, 40, 3000)]
                       for s in (1, 2, 3, 7, 40, 127, 128, 129, 300)] for n in (1, 2, 3, 5, 16, 17, 40, 300, 1000)] for g in (1, 2, 5, 8, 16, 40)])
    assert (need >= 16).all()
    for axis in range(4):
        assert (np.diff(need, axis=axis) >= 0).all(), f"axis {axis}"


def test_attend_formats():
    """Values of more bits than the keys are declined."""
    order = [M.QMM_IQ4_NL, M.QMM_Q8_0, M.QMM_F16]
    for i, k in enumerate(order):
        for j, v in enumerate(order):
            cache = struct(ktype=k, vtype=v, kstride=1 << 20, vstride=1 << 20)
            need = M.lib().qmm_kv_attend_workspace(C.addressof(cache), 7, 8, 3, 5)
            assert (need > 0) == (j <= i)
            a = dict(ATTEND, cache=C.addressof(cache), ws_bytes=0)
            assert M.lib().qmm_kv_attend(*a.values()) == (-5 if j <= i else -2)


def test_attend_workspace():
    def f(ntok, heads, nseq, width, **kw):
        cache = struct(**kw)
        return M.lib().qmm_kv_attend_workspace(C.addressof(cache), ntok, heads, nseq, width)

    assert M.lib().qmm_kv_attend_workspace(None, 1, 4, 1, 1) == 0
    assert f(-1, 8, 1, 1) == f(1, 6, 1, 1) == f(1, 8, -1, 1) == f(1, 8, 1, 0) == f(1, 8, 1, 1, head_dim=80) == f(1, 2048, 1, 1) == 0
    assert 0 < f(1, 4, 1, 1) <= f(8, 4, 8, 1) <= f(8, 4, 8, 64) <= f(64, 4, 64, 64) <= f(64, 8, 64, 64) <= f(1 << 12, 8, 1 << 12, 64)


# ------------------------------------------------------------------ the binding

def cache(kinds=("q8_0", "iq4_nl"), npages=5, heads=2, page=32, dim=64):
    """A KvCache of stand-ins."""
    class Tensor(Fake):
        def data_ptr(self):
            return 0x100000

        def __getitem__(self, i):
            return Tensor(self.shape[1:], self.dtype)
    import torch
    t = [Tensor((npages, heads, page, dim if k == "f16" else (R.FACTOR[k] + 2) * dim // 32), torch.float16 if k == "f16" else torch.uint8)
         for k in kinds]
    return M.KvCache(R.FORMATS[kinds[0]], R.FORMATS[kinds[1]], *t)


def test_cache_fields():
    c = cache(("f16", "q8_0"), npages=7, heads=3, page=48, dim=96)
    s = c._struct
    assert (s.npages, s.nheads, s.page_size, s.head_dim, s.kstride, s.vstride) == (7, 3, 48, 96, 3 * 48 * 192, 3 * 48 * 102)
    assert (c.npages, c.nheads, c.page_size, c.head_dim, c.width) == (7, 3, 48, 96, 288)


def test_cache_refuses():
    import torch
    u8, f16 = torch.uint8, torch.float16
    good = Fake((5, 2, 32, 68), u8)
    for bad in (Fake((5, 2, 32, 68), u8, device="cpu"), Fake((5, 2, 32, 68), f16), Fake((5, 2, 32, 67), u8), Fake((5, 2, 40, 68), u8),
                Fake((5, 2, 32, 34), u8), Fake((2, 32, 68), u8), Fake((0, 2, 32, 68), u8), Fake((5, 2, 8192, 68), u8), None,
                Fake((5, 2, 32, 68), u8, stride=(4352, 2176, 70, 1)), Fake((5, 2, 32, 68), u8, stride=(4000, 2176, 68, 1)),
                Fake((5, 2, 32, 68), u8, stride=(4352, 2200, 68, 1))):
        refused(M.KvCache, M.QMM_Q8_0, M.QMM_Q8_0, bad, good)
        refused(M.KvCache, M.QMM_Q8_0, M.QMM_Q8_0, good, bad)
    refused(M.KvCache, M.QMM_CB3, M.QMM_Q8_0, good, good)
    refused(M.KvCache, M.QMM_Q8_0, M.QMM_Q8_0, good, Fake((5, 2, 32, 68), u8, device="cuda:1"))
    refused(M.KvCache, M.QMM_Q8_0, M.QMM_Q8_0, good, Fake((5, 1, 32, 68), u8))
    refused(M.KvCache, M.QMM_Q8_0, M.QMM_Q8_0, good, Fake((5, 2, 32, 136), u8))
    refused(M.KvCache, M.QMM_F16, M.QMM_Q8_0, Fake((5, 2, 32, 80), f16), good)


def test_rows_refuse():
    import torch
    f32, f16, i32 = torch.float32, torch.float16, torch.int32
    c = cache()
    pages, lens, off = Fake((3, 4), i32), Fake((3,), i32), Fake((4,), i32)
    x = Fake((7, 128), f32)
    for fn in (M.qmm_kv_write, M.qmm_kv_read):
        ok = dict(k=x, v=x, seg_off=off)
        for bad in (dict(k=None, v=None), dict(k=Fake((7, 127), f32)), dict(v=Fake((6, 128), f32)), dict(v=Fake((7, 128), f16)),
                    dict(k=Fake((7, 128), torch.int32)), dict(k=Fake((7, 128), f32, device="cuda:1")), dict(k=Fake((7, 128), f32, device="cpu")),
                    dict(k=Fake((7, 128), f32, stride=(128, 2))), dict(k=Fake((7, 128), f32, stride=(100, 1))), dict(seg_off=None),
                    dict(seg_off=Fake((3,), i32)), dict(seg_off=Fake((4,), torch.int64)), dict(seg_off=Fake((4,), i32, device="cpu"))):
            refused(fn, c, pages, lens, **{**ok, **bad})
        for p in (Fake((3, 4), torch.int64), Fake((3, 4), i32, device="cpu"), Fake((12,), i32), Fake((3, 0), i32), Fake((2, 4), i32),
                  Fake((3, 4), i32, stride=(1, 3)), Fake((3, 4), i32, stride=(3, 1))):
            refused(fn, c, p, lens, **ok)
        for l in (Fake((2,), i32), Fake((3,), torch.int64), Fake((3,), i32, device="cpu"), Fake((3,), i32, stride=(2,))):
            refused(fn, c, pages, l, **ok)
    refused(M.qmm_kv_read, c, pages, lens, k=f32, seg_off=off)  # how many rows?
    refused(M.qmm_kv_read, c, pages, lens, k=f32, seg_off=off, ntok=-1)
    refused(M.qmm_kv_read, c, pages, lens, k=torch.int32)


def test_attend_refuses():
    import torch
    f32, i32 = torch.float32, torch.int32
    c = cache()
    pages, lens, off = Fake((3, 4), i32), Fake((3,), i32), Fake((4,), i32)
    ok = dict(q=Fake((7, 256), f32), seg_off=off, out=Fake((7, 256), f32), ws=Fake((1 << 24,), torch.uint8))
    for bad in (dict(q=Fake((7, 192), f32)), dict(q=Fake((7,), f32)), dict(q=Fake((7, 256), torch.float64)), dict(q=Fake((7, 256), f32, device="cpu")),
                dict(q=Fake((7, 256), f32, device="cuda:1")), dict(q=Fake((7, 0), f32)), dict(q=Fake((7, 256), f32, stride=(255, 1))),
                dict(out=Fake((7, 128), f32)), dict(out=Fake((6, 256), f32)), dict(out=torch.int32), dict(out=Fake((7, 256), f32, device="cpu")),
                dict(lse=Fake((7, 3), f32)), dict(lse=Fake((7, 4), torch.float64)), dict(ws=Fake((8,), torch.uint8)),
                dict(ws=Fake((1 << 24,), torch.int8)), dict(window=-1), dict(window=1 << 63), dict(seg_off=None), dict(seg_off=Fake((5,), i32))):
        a = {**ok, **bad}
        refused(M.qmm_kv_attend, a.pop("q"), c, pages, lens, **a)
    a = dict(ok)
    q = a.pop("q")
    refused(M.qmm_kv_attend, q, c, Fake((3, 4), torch.int64), lens, **a)
    refused(M.qmm_kv_attend, q, c, pages, Fake((4,), i32), **a)
