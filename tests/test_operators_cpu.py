"""The norm, routing, dispatch and adapter calls refuse bad arguments before anything is launched:
the C entry points by status, the binding by ValueError.  CPU only, no pointer is followed."""
import ctypes as C

import numpy as np
import pytest

import moe_expert_amd as M
from tests import operator_refs as R

FAKE = C.c_void_p(0x100000)
ODD = C.c_void_p(0x100001)
TWO = C.c_void_p(0x100002)


def call(fn, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    return getattr(M.lib(), fn)(*a.values())


NORM = dict(xtype=1, x=FAKE, ldx=64, rtype=2, res=FAKE, ldr=64, res_out=FAKE, ldro=64, w=FAKE, eps=1e-6, ntok=4, hidden=64,
            ytype=1, y=FAKE, ldy=64, yq=FAKE, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(xtype=0), -1), (dict(xtype=4), -1), (dict(rtype=9), -1), (dict(ytype=0), -1),
    (dict(y=None, yq=None, res_out=None), -1), (dict(hidden=0), -1), (dict(ntok=-1), -1), (dict(ldx=63), -1), (dict(ldr=63), -1),
    (dict(ldro=63), -1), (dict(ldy=63), -1), (dict(hidden=48), -1), (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(hidden=32800, ldx=32800, ldr=32800, ldro=32800, ldy=32800), -2), (dict(ntok=1 << 31), -2),
    (dict(x=TWO), -3), (dict(res=ODD), -3), (dict(res_out=ODD), -3), (dict(w=TWO), -3), (dict(y=TWO), -3), (dict(yq=TWO), -3),
    (dict(ntok=0, x=None, res=None, w=None, y=None, yq=None, res_out=None), 0),
])
def test_rmsnorm_rejects(kw, expect):
    assert call("qmm_rmsnorm", NORM, kw) == expect


DEQ = dict(xq=FAKE, k=64, ncols=3, otype=1, out=FAKE, ldo=64, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(xq=None), -1), (dict(out=None), -1), (dict(k=48), -1), (dict(k=0), -1), (dict(ncols=-1), -1), (dict(ldo=63), -1),
    (dict(otype=3), -1), (dict(ncols=1 << 31), -2), (dict(xq=TWO), -3), (dict(out=TWO), -3), (dict(ncols=0, xq=None), 0),
])
def test_dequantize_q8_1_rejects(kw, expect):
    assert call("qmm_dequantize_q8_1", DEQ, kw) == expect


ROUTE = dict(ltype=1, logits=FAKE, ldl=64, bias=FAKE, ntok=4, nexperts=64, score=0, ngroups=8, topk_groups=3, group_top=2, topk=6,
             scale=1.0, ids=FAKE, weights=FAKE, flags=1, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(logits=None), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(ltype=0), -1), (dict(score=2), -1),
    (dict(flags=2), -1), (dict(ntok=-1), -1), (dict(nexperts=0), -1), (dict(ldl=63), -1), (dict(ngroups=0), -1), (dict(ngroups=7), -1),
    (dict(topk_groups=0), -1), (dict(topk_groups=9), -1), (dict(topk=0), -1), (dict(topk=25), -1), (dict(group_top=0), -1),
    (dict(group_top=3), -1), (dict(ngroups=64, topk_groups=10, group_top=2), -1), (dict(nexperts=1032, ldl=1032), -2),
    (dict(nexperts=1024, ldl=1024, ngroups=128), -2), (dict(nexperts=1024, ldl=1024, topk=65), -2), (dict(ntok=1 << 31), -2),
    (dict(logits=TWO), -3), (dict(bias=TWO), -3), (dict(ids=TWO), -3), (dict(weights=TWO), -3), (dict(ntok=0, logits=None), 0),
])
def test_route_rejects(kw, expect):
    assert call("qmm_moe_route", ROUTE, kw) == expect


DISP = dict(ids=FAKE, ntok=4, topk=8, nexperts=64, sorted_tok=FAKE, row_idx=FAKE, expert_off=FAKE, ge=FAKE, go=FAKE, ws=FAKE,
            ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(ids=None), -1), (dict(sorted_tok=None), -1), (dict(row_idx=None), -1), (dict(expert_off=None), -1), (dict(ge=None), -1),
    (dict(go=None), -1), (dict(ws=None), -1), (dict(ntok=-1), -1), (dict(topk=0), -1), (dict(nexperts=0), -1), (dict(nexperts=1025), -2),
    (dict(topk=65), -2), (dict(ntok=1 << 28), -2), (dict(ids=TWO), -3), (dict(row_idx=TWO), -3), (dict(ws=TWO), -3),
    (dict(ws_bytes=0), -5),
])
def test_dispatch_rejects(kw, expect):
    assert call("qmm_moe_dispatch", DISP, kw) == expect


def test_dispatch_workspace():
    f = M.lib().qmm_moe_dispatch_workspace
    assert f(-1, 8, 64) == f(4, 0, 64) == f(4, 8, 0) == f(4, 65, 64) == f(4, 8, 1025) == f(1 << 28, 8, 64) == 0
    assert 0 < f(1, 1, 1) <= f(8192, 8, 128) <= f(1 << 24, 64, 1024)


LORA = dict(xtype=2, x=FAKE, ldx=64, ntok=4, k=64, a=FAKE, b=FAKE, ranks=FAKE, scales=FAKE, na=2, max_rank=16, seg_off=FAKE,
            seg_adapter=FAKE, nseg=1, base=FAKE, ldb=100, y=FAKE, ldy=100, nrows=100, ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), -1), (dict(a=None), -1), (dict(b=None), -1), (dict(ranks=None), -1), (dict(scales=None), -1), (dict(seg_off=None), -1),
    (dict(seg_adapter=None), -1), (dict(base=None), -1), (dict(y=None), -1), (dict(ws=None), -1), (dict(xtype=3), -1), (dict(ntok=-1), -1),
    (dict(k=48, ldx=48), -1), (dict(k=0), -1), (dict(ldx=56), -1), (dict(na=0), -1), (dict(max_rank=12), -1), (dict(max_rank=0), -1),
    (dict(nseg=-1), -1), (dict(nrows=0), -1), (dict(ldb=99, base=C.c_void_p(0x200000)), -1), (dict(ldy=99), -1), (dict(ldb=104), -1),
    (dict(k=32800, ldx=32800), -2), (dict(max_rank=264), -2), (dict(ntok=1 << 31), -2), (dict(nrows=1 << 31, ldb=1 << 31, ldy=1 << 31), -2),
    (dict(x=C.c_void_p(0x100008)), -3), (dict(ldx=68), -3), (dict(a=C.c_void_p(0x100008)), -3), (dict(b=TWO), -3), (dict(y=TWO, base=FAKE), -3),
    (dict(base=TWO), -3), (dict(ranks=TWO), -3), (dict(ws=C.c_void_p(0x100008)), -3), (dict(ws_bytes=16), -5), (dict(ntok=0, x=None), 0),
    (dict(nseg=0, seg_off=None, seg_adapter=None), 0),
])
def test_lora_rejects(kw, expect):
    assert call("qmm_lora", LORA, kw) == expect


def test_lora_workspace():
    f = M.lib().qmm_lora_workspace
    assert f(-1, 16) == f(8, 0) == f(8, 12) == f(8, 264) == f(1 << 31, 16) == 0
    assert 0 < f(1, 8) <= f(8192, 16) <= f(8192, 256)


# ------------------------------------------------------------------ the binding

class Fake:
    """A GPU tensor as the binding's checks see it; its pointer must not be read."""

    def __init__(self, shape, dtype, device="cuda:0", stride=None):
        import torch
        self.shape, self.dtype, self.device = tuple(shape), dtype, torch.device(device)
        self.is_cuda = self.device.type == "cuda"
        self._stride = stride

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        import torch
        return torch.empty((), dtype=self.dtype).element_size()

    def stride(self):
        if self._stride:
            return self._stride
        return tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def is_contiguous(self):
        return self._stride is None

    def data_ptr(self):
        raise AssertionError("the binding must refuse this call before reading a pointer")


def refused(fn, *args, **kw):
    with pytest.raises(ValueError):
        fn(*args, **kw)


def test_binding_refuses_bad_norm_tensors():
    import torch
    f32, f16, u8 = torch.float32, torch.float16, torch.uint8
    x, w, y, yq = Fake((4, 64), f32), Fake((64,), f32), Fake((4, 64), f16), Fake((4, 72), u8)
    N = M.qmm_rmsnorm
    refused(N, x, w, 1e-6)                                               # no output
    refused(N, Fake((64,), f32), w, 1e-6, y=y)                           # one dimension
    refused(N, Fake((4, 64), f32, "cpu"), w, 1e-6, y=y)
    refused(N, Fake((4, 64), torch.float64), w, 1e-6, y=y)
    refused(N, x, Fake((63,), f32), 1e-6, y=y)
    refused(N, x, Fake((64,), f16), 1e-6, y=y)
    refused(N, x, w, 1e-6, y=Fake((4, 65), f16))
    refused(N, x, w, 1e-6, y=Fake((3, 64), f16))
    refused(N, x, w, 1e-6, y=Fake((4, 64), f16, stride=(64, 2)))
    refused(N, x, w, 1e-6, y=Fake((4, 64), f16, stride=(0, 1)))          # rows that overlap
    refused(N, Fake((4, 64), f32, stride=(0, 1)), w, 1e-6, y=y)
    refused(N, x, w, 1e-6, y=Fake((4, 64), f16, "cuda:1"))
    refused(N, x, w, 1e-6, yq=Fake((4, 71), u8))
    refused(N, Fake((4, 48), f32), Fake((48,), f32), 1e-6, yq=yq)
    refused(N, x, w, 1e-6, y=y, res=Fake((4, 63), f32))
    refused(N, x, w, 1e-6, y=y, res=Fake((4, 64), f32), res_out=Fake((4, 64), f16))
    D = M.qmm_dequantize_q8_1
    refused(D, yq, 48)
    refused(D, yq, 96)
    refused(D, yq, 64, out=Fake((4, 64), torch.bfloat16))
    refused(D, yq, 64, out=Fake((4, 32), f32))


def test_binding_refuses_bad_routing_tensors():
    import torch
    f32, i32 = torch.float32, torch.int32
    z = Fake((4, 64), f32)
    T = M.qmm_moe_route
    refused(T, Fake((4, 64), i32), 2)
    refused(T, Fake((4, 64), f32, "cpu"), 2)
    refused(T, Fake((4, 64), f32, stride=(1, 4)), 2)
    refused(T, z, 0)
    refused(T, z, (1 << 32) + 1)
    refused(T, z, 2, bias=Fake((63,), f32))
    refused(T, z, 2, ids=Fake((4, 2), torch.int64))
    refused(T, z, 2, ids=Fake((3, 2), i32))
    refused(T, z, 2, ids=Fake((4, 2), i32), weights=Fake((4, 1), f32))
    ids = Fake((4, 2), i32)
    P = M.qmm_moe_dispatch
    good = dict(sorted_tok=Fake((8,), i32), row_idx=Fake((4, 2), i32), expert_off=Fake((65,), i32), group_expert=Fake((8,), i32),
                group_off=Fake((9,), i32), ws=Fake((1 << 20,), torch.uint8))
    refused(P, Fake((8,), i32), 64, **good)
    refused(P, Fake((4, 2), torch.int64), 64, **good)
    refused(P, Fake((4, 2), i32, stride=(1, 4)), 64, **good)
    refused(P, ids, 0, **good)
    refused(P, ids, 1 << 32, **good)
    for name, bad in (("sorted_tok", Fake((7,), i32)), ("row_idx", Fake((3, 2), i32)), ("expert_off", Fake((64,), i32)),
                      ("group_expert", Fake((7,), i32)), ("group_off", Fake((8,), i32)), ("group_off", None),
                      ("ws", Fake((1,), torch.uint8)), ("expert_off", Fake((65,), i32, "cuda:1"))):
        refused(P, ids, 64, **dict(good, **{name: bad}))


def test_binding_refuses_bad_adapter_tensors():
    import torch
    f32, f16, i32 = torch.float32, torch.float16, torch.int32
    good = dict(x=Fake((4, 64), f16), a=Fake((2, 16, 64), f16), b=Fake((2, 100, 16), f16), ranks=Fake((2,), i32), scales=Fake((2,), f32),
                seg_off=Fake((2,), i32), seg_adapter=Fake((1,), i32), y=Fake((4, 100), f32), base=Fake((4, 100), f32),
                ws=Fake((1 << 20,), torch.uint8))
    for name, bad in (("x", Fake((4, 64), torch.bfloat16)), ("x", Fake((4, 32), f16)), ("x", Fake((64,), f16)), ("a", Fake((2, 16, 32), f16)),
                      ("a", Fake((2, 16, 64), torch.int16)), ("a", Fake((2, 16, 64), f16, stride=(1024, 1, 16))), ("b", Fake((2, 100, 8), f16)),
                      ("b", Fake((1, 100, 16), f16)), ("ranks", Fake((1,), i32)), ("scales", Fake((2,), f16)), ("seg_off", Fake((1,), i32)),
                      ("seg_adapter", Fake((1,), torch.int64)), ("y", Fake((4, 100), f16)), ("y", Fake((4, 99), f32)),
                      ("y", Fake((4, 100), f32, stride=(0, 1))), ("base", Fake((3, 100), f32)), ("ws", Fake((16,), torch.uint8)),
                      ("scales", Fake((2,), f32, "cuda:1")), ("ranks", Fake((2,), i32, "cpu"))):
        refused(M.qmm_lora, **dict(good, **{name: bad}))


# ------------------------------------------------------------------ the references themselves

def test_reference_route_by_hand():
    z = np.array([[0.0, 2.0, 2.0, -np.inf], [-np.inf] * 4, [np.nan, 1.0, -np.inf, -np.inf]], np.float32)
    ids, w, _ = R.route(z, 2, True)
    assert ids.tolist() == [[1, 2], [-1, -1], [1, -1]]
    assert np.allclose(w, [[0.5, 0.5], [0, 0], [1, 0]])
    ids, w, _ = R.route(z, 3, True, renorm=False, scale=2.0)
    assert ids.tolist()[0] == [1, 2, 0] and np.isclose(w[0].sum(), 2.0)
    ids, _, _ = R.route(np.array([[3.0, -9.0, 2.5, 2.4]], np.float32), 1, False, ngroups=2, topk_groups=1, group_top=2)
    assert ids.tolist() == [[2]]  # the runs' sums, 0.953 + 0.000 and 0.924 + 0.917


def test_reference_dispatch_by_hand():
    st, ri, off, ge, go = R.dispatch(np.array([[2, 0], [-1, 2], [0, 7]], np.int32), 4)
    assert st.tolist() == [0, 2, 0, 1, -1, -1] and ri.tolist() == [[2, 0], [-1, 3], [1, -1]]
    assert off.tolist() == [0, 2, 2, 4, 4] and ge.tolist() == [0, 2, -1, -1] and go.tolist() == [0, 2, 4, 4, 4]
