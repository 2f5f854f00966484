"""GPU tests of the adapters (qmm_lora) against the 64-bit reference, within its derived bound."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import operator_refs as R
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu


def inputs(seed, ntok, k, nrows, max_rank, lens, adapters, na, xt="f16", ranks=None, xscale=1.0):
    """Random inputs; the table's rows and columns past each adapter's rank hold NaN."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((ntok, k)) * xscale).astype(np.float16 if xt == "f16" else np.float32)
    a = (rng.standard_normal((na, max_rank, k)) / np.sqrt(k)).astype(np.float16)
    b = rng.standard_normal((na, nrows, max_rank)).astype(np.float16)
    ranks = rng.integers(1, max_rank + 1, na).astype(np.int32) if ranks is None else np.asarray(ranks, np.int32)
    for i, r in enumerate(ranks):
        r = min(max(int(r), 0), max_rank)
        a[i, r:] = np.nan
        b[i, :, r:] = np.nan
    scales = rng.uniform(-2, 2, na).astype(np.float32)
    seg_off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    base = rng.standard_normal((ntok, nrows)).astype(np.float32)
    return x, a, b, ranks, scales, seg_off, np.asarray(adapters, np.int32), base


def check(arrays, y, sentinel=None):
    want, bound, written = R.lora(*arrays)
    err = np.abs(y.astype(np.float64) - want)
    ok = err <= bound
    assert ok[written].all(), f"{(~ok[written]).sum()} outside, worst {np.nanmax((err / bound)[written])}"
    if sentinel is not None:
        assert (y[~written] == sentinel).all()


def run(arrays, in_place=False):
    import torch
    x, a, b, ranks, scales, seg_off, adapters, base = arrays
    bt = dev(base)
    y = bt if in_place else torch.full_like(bt, 5.0)
    M.qmm_lora(dev(x), dev(a), dev(b), dev(ranks), dev(scales), dev(seg_off), dev(adapters), y, base=None if in_place else bt)
    return host(y)


SHAPES = [  # ntok, k, nrows, max_rank, segment lengths, adapters, table
    (1, 32, 1, 8, [1], [0], 1),
    (1, 2560, 8192, 16, [1], [2], 4),
    (8, 2560, 4096, 16, [1] * 8, [0, 3, 1, -1, 2, 2, 7, 5], 8),
    (8, 2560, 1000, 64, [8], [1], 2),
    (5, 64, 77, 24, [2, 0, 3], [1, 0, 2], 3),
    (33, 96, 129, 40, [16, 1, 16], [0, 1, 0], 2),
    (64, 2560, 513, 16, [64], [0], 1),
    (130, 1024, 300, 8, [65, 65], [1, 0], 2),
    (517, 2560, 640, 64, [100, 1, 0, 200, 3, 150, 63], [3, 2, 1, -1, 0, 3, 9], 4),
    (300, 6144, 257, 128, [33, 267], [0, 1], 2),
    (70, 160, 65, 256, [7, 63], [1, 0], 2),
    (1000, 512, 1024, 32, [1] * 100 + [900], [i % 5 for i in range(101)], 5),
    (200, 32, 30001, 16, [200], [0], 1),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}r{s[3]}")
@pytest.mark.parametrize("xt", ["f16", "f32"])
def test_lora(shape, xt):
    ntok, k, nrows, r, lens, adapters, na = shape
    print(f"lora {ntok} x {k} -> {nrows} rank {r} {xt}", flush=True)
    arrays = inputs(ntok + k + r, ntok, k, nrows, r, lens, adapters, na, xt)
    y = run(arrays)
    check(arrays, y)
    assert np.array_equal(run(arrays, in_place=True), y)
    assert np.array_equal(run(arrays), y)  # the same bits again


@pytest.mark.parametrize("xt", ["f16", "f32"])
def test_lora_ranks_and_segments_at_their_edges(xt):
    """Ranks of 0, below 0 and above the table's; tokens of no segment before, between and after
    the segments keep what is there; offsets outside the tokens are clamped; no segments at all."""
    import torch
    x, a, b, _, scales, _, _, base = inputs(4, 50, 320, 200, 16, [50], [0], 5, xt, ranks=[16, 16, 16, 16, 16])
    ranks = np.array([0, -3, 99, 1, 15], np.int32)
    seg_off = np.array([4, 4, 20, 30, 31, 48], np.int32)
    adapters = np.array([0, 2, 1, 4, 3], np.int32)
    arrays = (x, a, b, ranks, scales, seg_off, adapters, base)
    y = run(arrays)
    check(arrays, y, sentinel=5.0)
    off = np.array([-5, 10, 40, 70], np.int32)
    arrays = (x, a, b, ranks, scales, off, np.array([2, 4, 2], np.int32), base)
    check(arrays, run(arrays), sentinel=5.0)
    none = (x, a, b, ranks, scales, np.zeros(1, np.int32), np.empty(0, np.int32), base)
    assert (run(none) == 5.0).all()


@pytest.mark.parametrize("xt", ["f16", "f32"])
@pytest.mark.parametrize("xscale", [1e-6, 3e3])
def test_lora_magnitudes(xt, xscale):
    """Inner values far below and above binary16's range keep their precision."""
    arrays = list(inputs(9, 70, 640, 100, 32, [1, 69], [1, 0], 2, xt, xscale=xscale))
    arrays[1] = (arrays[1].astype(np.float32) * 50).astype(np.float16)
    arrays[7] = np.zeros_like(arrays[7])
    check(arrays, run(tuple(arrays)))


@pytest.mark.parametrize("xt", ["f16", "f32"])
def test_lora_infinities_stay_in_their_rows(xt):
    arrays = inputs(11, 40, 320, 90, 16, [3, 37], [1, 0], 2, xt, ranks=[16, 16])
    clean = run(arrays)
    arrays[0][2, 5] = np.inf
    arrays[0][20, 7] = np.nan
    y = run(arrays)
    for t in (2, 20):
        assert not np.isfinite(y[t]).any()
    keep = [t for t in range(40) if t not in (2, 20)]
    assert np.array_equal(y[keep], clean[keep])


def test_lora_strides_stream_and_graph():
    """x, y and base as views of wider tensors at odd places; a captured graph replayed on new x; a
    stream given."""
    import torch
    arrays = inputs(13, 100, 256, 333, 16, [10, 90], [0, 1], 2)
    x, a, b, ranks, scales, seg_off, adapters, base = [dev(v) for v in arrays]
    want = torch.from_numpy(run(arrays)).cuda()
    xw = torch.zeros(100, 256 + 24, dtype=torch.float16, device="cuda")
    xw[:, 8:264] = x
    yw, bw = torch.full((100, 340), 5.0, device="cuda"), torch.zeros(100, 351, device="cuda")
    bw[:, 11:344] = base
    M.qmm_lora(xw[:, 8:264], a, b, ranks, scales, seg_off, adapters, yw[:, 3:336], base=bw[:, 11:344])
    assert torch.equal(yw[:, 3:336], want) and (yw[:, :3] == 5).all() and (yw[:, 336:] == 5).all()
    y = torch.empty_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    M.qmm_lora(x, a, b, ranks, scales, seg_off, adapters, y, base=base, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, want)
    ws = torch.empty(M.qmm_lora_workspace(100, 16), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.qmm_lora(x, a, b, ranks, scales, seg_off, adapters, y, base=base, ws=ws)
    for i in range(3):
        x.mul_(-0.5)
        want = M.qmm_lora(x, a, b, ranks, scales, seg_off, adapters, torch.empty_like(y), base=base)
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_lora_offsets_past_32_bits():
    """Output rows that lie gigabytes apart, and an adapter table of over 4 GiB."""
    import torch
    arrays = inputs(17, 3, 64, 100, 8, [3], [0], 1)
    x, a, b, ranks, scales, seg_off, adapters, base = [dev(v) for v in arrays]
    ld = (1 << 30) + 64
    y = torch.empty(2 * ld + 100, device="cuda").as_strided((3, 100), (ld, 1))
    M.qmm_lora(x, a, b, ranks, scales, seg_off, adapters, y, base=base)
    check(arrays, host(y.contiguous()))
    del y
    na, r, k, rows = 1100, 64, 32768, 8
    big = torch.zeros(na, r, k, dtype=torch.float16, device="cuda")
    rng = np.random.default_rng(1)
    last = (rng.standard_normal((r, k)) / 181).astype(np.float16)
    big[na - 1] = dev(last)
    b1 = (rng.standard_normal((rows, r))).astype(np.float16)
    bb = torch.zeros(na, rows, r, dtype=torch.float16, device="cuda")
    bb[na - 1] = dev(b1)
    x1 = rng.standard_normal((20, k)).astype(np.float16)
    base1 = np.zeros((20, rows), np.float32)
    rk, sc = torch.full((na,), r, dtype=torch.int32, device="cuda"), torch.ones(na, device="cuda")
    y1 = torch.empty(20, rows, device="cuda")
    M.qmm_lora(dev(x1), big, bb, rk, sc, dev(np.array([0, 20], np.int32)), dev(np.array([na - 1], np.int32)), y1, base=dev(base1))
    one = (x1, last[None], b1[None], np.array([r]), np.ones(1), np.array([0, 20]), np.array([0]), base1)
    check(one, host(y1))


@pytest.mark.parametrize("nseg", [64, 65, 256, 700])
def test_lora_many_segments(nseg):
    """More segments than one step, or one round, of the kernels' scan takes; empty ones among them."""
    rng = np.random.default_rng(nseg)
    lens = rng.integers(0, 4, nseg)
    arrays = inputs(nseg, int(lens.sum()), 128, 200, 16, lens, rng.integers(-1, 6, nseg), 6)
    check(arrays, run(arrays))


def test_lora_given_stream_allocates_there():
    """A call on a given stream takes its workspace and nothing else from the caller's stream: memory
    that pending work of the caller's stream has given back is not touched."""
    import torch
    arrays = inputs(21, 300, 512, 640, 16, [300], [0], 1)
    x, a, b, ranks, scales, seg_off, adapters, base = [dev(v) for v in arrays]
    want = M.qmm_lora(x, a, b, ranks, scales, seg_off, adapters, torch.empty_like(base), base=base)
    side = torch.cuda.Stream()
    y = torch.empty_like(base)
    torch.cuda.synchronize()
    n = M.qmm_lora_workspace(300, 16)
    for _ in range(20):
        junk = torch.empty(n, dtype=torch.uint8, device="cuda")
        for _ in range(4):
            junk.fill_(255)  # still running when its memory is given back
        del junk
        M.qmm_lora(x, a, b, ranks, scales, seg_off, adapters, y, base=base, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
