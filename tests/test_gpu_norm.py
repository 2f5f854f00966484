"""GPU tests of the norm with the residual's addition (qmm_rmsnorm) and of the q8_1 values
(qmm_dequantize_q8_1) against 64-bit references: r and q8_1 bit for bit, y within its bound."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import operator_refs as R
from tests.gpu_util import host

pytestmark = pytest.mark.gpu

TYPES = ["f32", "f16", "bf16"]


def dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def values(t):
    return host(t.float())


def rows(rng, ntok, hidden, name, pad=0, offset=0, scale=1.0):
    """[ntok, hidden] of the type; a view with row stride hidden + pad that starts `offset` elements
    into its storage."""
    import torch
    ld = hidden + pad
    store = torch.full((offset + ntok * ld,), 7.0, dtype=dtype(name), device="cuda")
    v = store[offset:].view(ntok, ld)[:, :hidden]
    v.copy_(torch.from_numpy((rng.standard_normal((ntok, hidden)) * scale).astype(np.float32)))
    return v


def check(x, res, w, eps, y, yq, res_out, ytype):
    import torch
    ntok, hidden = x.shape
    r64, y64 = R.rmsnorm(values(x), None if res is None else values(res), host(w), eps)
    if res_out is not None:
        want = x.float() if res is None else x.float() + res.float()
        assert torch.equal(res_out, want.to(res_out.dtype))
    err = np.abs(values(y).astype(np.float64) - y64)
    bound = R.rmsnorm_bound(y64, hidden, ytype)
    assert (err <= bound).all(), f"{(err > bound).sum()} outside, worst {np.max(err / bound)}"
    if yq is not None and ytype == "f32":
        assert torch.equal(yq, M.qmm_quantize_q8_1(y.contiguous()))


@pytest.mark.parametrize("ntok,hidden", [(1, 1), (3, 7), (1, 31), (2, 32), (5, 33), (4, 64), (1, 2560), (8, 2560), (700, 2560),
                                         (517, 1001), (3, 4100), (700, 4096), (2, 8192), (300, 6144), (1, 12288), (3, 20000),
                                         (2, 32768), (3, 32767), (70000, 32), (1200, 96), (1, 544)])
@pytest.mark.parametrize("xt,rt", [("f32", "f32"), ("f16", ""), ("bf16", "f16")])
def test_norm_sizes(ntok, hidden, xt, rt):
    """Row lengths from 1 to the limit, one row to 70000, with the float32 and (where the row is
    whole blocks) the q8_1 output."""
    import torch
    print(f"norm {ntok} x {hidden} {xt} {rt}", flush=True)
    rng = np.random.default_rng(10 * hidden + ntok)
    x = rows(rng, ntok, hidden, xt)
    res = rows(rng, ntok, hidden, rt) if rt else None
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(hidden)).astype(np.float32)).cuda()
    res_out = torch.empty_like(x if res is None else res)
    y, yq, _ = M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=res_out, y=torch.float32, yq=True if hidden % 32 == 0 else None)
    check(x, res, w, 1e-6, y, yq, res_out, "f32")


@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("rt", [""] + TYPES)
@pytest.mark.parametrize("yt", TYPES)
def test_norm_types(xt, rt, yt):
    """Every combination of input, residual and output types."""
    import torch
    print(f"norm types {xt} {rt} {yt}", flush=True)
    rng = np.random.default_rng(77)
    for ntok, hidden in ((5, 2560), (3, 1003)):
        x = rows(rng, ntok, hidden, xt)
        res = rows(rng, ntok, hidden, rt) if rt else None
        w = torch.from_numpy(rng.standard_normal(hidden).astype(np.float32)).cuda()
        res_out = torch.empty(ntok, hidden, dtype=dtype(rt), device="cuda") if rt else None
        y, yq, _ = M.qmm_rmsnorm(x, w, 1e-5, res=res, res_out=res_out, y=dtype(yt), yq=True if hidden % 32 == 0 else None)
        check(x, res, w, 1e-5, y, yq, res_out, yt)


@pytest.mark.parametrize("hidden,pad,offset", [(2560, 8, 0), (2560, 3, 0), (2560, 0, 1), (1001, 7, 3), (96, 1, 5), (4096, 16, 8)])
@pytest.mark.parametrize("name", ["f32", "f16"])
def test_norm_strides_and_alignment(hidden, pad, offset, name):
    """Row strides and starts that are not 16-byte aligned, in inputs and outputs; what lies between
    the output rows stays."""
    import torch
    print(f"norm strides {hidden}+{pad} at {offset} {name}", flush=True)
    rng = np.random.default_rng(hidden + pad)
    ntok = 9
    x, res = rows(rng, ntok, hidden, name, pad, offset), rows(rng, ntok, hidden, name, pad, offset)
    y, res_out = rows(rng, ntok, hidden, name, pad, offset), rows(rng, ntok, hidden, name, pad, offset)
    w = torch.from_numpy(rng.standard_normal(hidden + offset).astype(np.float32)).cuda()[offset:]
    M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=res_out, y=y)
    check(x, res, w, 1e-6, y, None, res_out, name)
    if pad:
        for t in (y, res_out):
            gap = t.as_strided((ntok - 1, pad), (hidden + pad, 1), t.storage_offset() + hidden)
            assert (gap == 7.0).all()


def test_norm_in_place():
    """The residual updated in place, the norm written over x, and the residual alone."""
    import torch
    rng = np.random.default_rng(3)
    for ntok, hidden in ((1, 2560), (600, 2560), (4, 1001)):
        x, res = rows(rng, ntok, hidden, "f32"), rows(rng, ntok, hidden, "f32")
        w = torch.from_numpy(rng.standard_normal(hidden).astype(np.float32)).cuda()
        want, _, r = M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=torch.empty_like(res), y=torch.float32)
        x2, res2 = x.clone(), res.clone()
        M.qmm_rmsnorm(x2, w, 1e-6, res=res2, res_out=res2, y=x2)
        assert torch.equal(x2, want) and torch.equal(res2, r)
        alone = torch.empty_like(res)
        M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=alone)
        assert torch.equal(alone, r)


def test_norm_values_out_of_the_ordinary():
    """Zero rows, rows of infinities and NaN, rows whose squares pass binary32's range or fall under
    it: each row as its definition has it, no row touching another."""
    import torch
    hidden = 2560
    x = torch.ones(8, hidden, device="cuda")
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 9] = float("nan")
    x[3] = 1e30
    x[4] = 1e-30
    x[5] = -torch.finfo(torch.float32).max
    w = torch.full((hidden,), 2.0, device="cuda")
    y, yq, _ = M.qmm_rmsnorm(x, w, 1e-6, y=torch.float32, yq=True)
    y = host(y)
    one = 2.0 / np.sqrt(1 + 1e-6)
    assert (y[0] == 0).all()
    assert np.isnan(y[1, 5]) and (np.delete(y[1], 5) == 0).all()
    assert np.isnan(y[2]).all()
    assert (y[3] == 0).all() and (y[5] == 0).all()
    assert np.allclose(y[4], 2e-27, rtol=1e-5)
    assert np.allclose(y[6:], one, rtol=1e-6)
    assert torch.equal(yq, M.qmm_quantize_q8_1(torch.from_numpy(y).cuda()))


def test_norm_offsets_past_32_bits():
    """Rows that lie gigabytes apart."""
    import torch
    rng = np.random.default_rng(8)
    hidden, ld = 2560, (1 << 31) + 64
    store = torch.empty(2 * ld + hidden, dtype=torch.float16, device="cuda")
    x = store.as_strided((3, hidden), (ld, 1))
    x.copy_(torch.from_numpy(rng.standard_normal((3, hidden)).astype(np.float32)))
    out = torch.empty_like(store).as_strided((3, hidden), (ld, 1))
    w = torch.ones(hidden, device="cuda")
    M.qmm_rmsnorm(x, w, 1e-6, y=out)
    want, _, _ = M.qmm_rmsnorm(x.contiguous(), w, 1e-6, y=torch.float16)
    assert torch.equal(out.contiguous(), want)


def test_norm_no_rows():
    import torch
    y, yq, _ = M.qmm_rmsnorm(torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda"), 1e-6, y=torch.float16, yq=True)
    assert y.shape == (0, 64) and yq.shape == (0, 72)


@pytest.mark.parametrize("ncols,k", [(1, 32), (3, 96), (7, 2560), (300, 6144)])
@pytest.mark.parametrize("name", ["f32", "f16"])
def test_dequantize_q8_1(ncols, k, name):
    """d * q exactly (float32), or rounded once (float16); also into rows of a wider tensor."""
    import torch
    rng = np.random.default_rng(k)
    x = torch.from_numpy((rng.standard_normal((ncols, k)) * np.exp2(rng.integers(-12, 12, (ncols, 1)))).astype(np.float32)).cuda()
    xq = M.qmm_quantize_q8_1(x)
    b = host(xq).reshape(ncols, k // 32, 36)
    d = b[:, :, :2].copy().view(np.float16).astype(np.float64)
    want = (d * b[:, :, 4:].copy().view(np.int8)).reshape(ncols, k)
    got = M.qmm_dequantize_q8_1(xq, k, out=dtype(name))
    kind = np.float32 if name == "f32" else np.float16
    assert np.array_equal(host(got), want.astype(kind))
    wide = torch.full((ncols, k + 5), 3.0, dtype=dtype(name), device="cuda")
    M.qmm_dequantize_q8_1(xq, k, out=wide[:, 1:k + 1])
    assert torch.equal(wide[:, 1:k + 1], got) and (wide[:, 0] == 3).all() and (wide[:, k + 1:] == 3).all()


def test_norm_on_another_stream_and_in_a_graph():
    """A stream given, a current stream other than the default, and replays of a captured graph
    between eager work: the eager result each time."""
    import torch
    rng = np.random.default_rng(5)
    x, res = rows(rng, 64, 2560, "f32"), rows(rng, 64, 2560, "f16")
    w = torch.ones(2560, device="cuda")
    want = M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=torch.empty_like(res), y=torch.float16, yq=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=got[2], y=got[0], yq=got[1], stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=got[2], y=got[0], yq=got[1])
    for i in range(3):
        x.add_(0.25 * i)
        want = M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=torch.empty_like(res), y=torch.float16, yq=True)
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
