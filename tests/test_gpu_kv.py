"""GPU tests of the paged key-value cache's writes and reads (qmm_kv_write, qmm_kv_read): the bytes of every
format bit for bit, and the values they read back as."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import kv_refs as R
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

PAIRS = [("q8_0", "iq4_nl"), ("f16", "q8_0"), ("iq4_nl", "f16"), ("iq4_nl", "q8_0")]


def dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def empty_cache(kind, npages, heads, page, dim, fill):
    """A raw cache tensor of bytes `fill`, as its format's dtype."""
    import torch
    row = 2 * dim if kind == "f16" else (R.FACTOR[kind] + 2) * dim // 32
    t = torch.full((npages, heads, page, row), fill, dtype=torch.uint8, device="cuda")
    return t.view(torch.float16) if kind == "f16" else t


def expected(raw, kind, x, seq, pos, pages, heads, page, dim):
    """The cache's bytes (numpy, a copy of `raw`) after the rows x [ntok, heads * dim] are written."""
    want = raw.copy()
    npages = raw.shape[0]
    with np.errstate(all="ignore"):
        for t in range(len(seq)):
            if seq[t] < 0 or pos[t] < 0 or pos[t] >= pages.shape[1] * page:
                continue
            pg, at = pages[seq[t], pos[t] // page], pos[t] % page
            if not 0 <= pg < npages:
                continue
            for h in range(heads):
                row = x[t, h * dim:(h + 1) * dim].astype(np.float32)
                if kind == "f16":
                    want[pg, h, at] = row.astype(np.float16)
                    continue
                code, d = R.quantize(row[None], kind)
                one = R.chunk_bytes(code, d, kind)
                fb = dim // 32 * R.FACTOR[kind]
                flat = want[pg, h].reshape(-1)
                flat[at * fb:(at + 1) * fb] = one[:fb]
                flat[page * fb + at * (dim // 16):page * fb + (at + 1) * (dim // 16)] = one[fb:]
    return want


def raw_bytes(t):
    return host(t).view(np.uint8)


def check(kinds, x, lens, seg_off, page, dim, heads, name="f32", pages=None, npages=None, missing=-1):
    """Write x (numpy float32, of the type's values) over a cache of 0xA5 and read the same rows back."""
    import torch
    rng = np.random.default_rng(len(lens))
    ntok = x.shape[0]
    if pages is None:
        pages, npages = R.tables(rng, lens, page, missing=missing)
    raws = [empty_cache(k, npages, heads, page, dim, 0xA5) for k in kinds]
    before = [host(r) for r in raws]
    cache = M.KvCache(R.FORMATS[kinds[0]], R.FORMATS[kinds[1]], *raws)
    xd = [dev(v).to(dtype(name)) for v in (x, -x[:, ::-1].copy())]
    off = None if seg_off is None else dev(np.asarray(seg_off, np.int32))
    pd, ld = dev(pages), dev(np.asarray(lens, np.int32))
    M.qmm_kv_write(cache, pd, ld, xd[0], xd[1], seg_off=off)
    seq, pos = R.positions(seg_off, lens, ntok, len(lens))
    sides = []
    for kind, raw, was, xs in zip(kinds, raws, before, xd):
        want = expected(was, kind, host(xs.float()), seq, pos, pages, heads, page, dim)
        assert np.array_equal(raw_bytes(raw), want.view(np.uint8)), f"{kind} bytes differ"
        sides.append(want)
    for out in ("f32", "f16", "bf16"):
        into = [torch.full((ntok, heads * dim), 7.0, dtype=dtype(out), device="cuda") for _ in range(2)]
        M.qmm_kv_read(cache, pd, ld, k=into[0], v=into[1], seg_off=off)
        for kind, want, got in zip(kinds, sides, into):
            ref = np.full((ntok, heads, dim), 7.0)
            for t in range(ntok):
                if seq[t] < 0:
                    continue
                ref[t] = 0.0
                if 0 <= pos[t] < pages.shape[1] * page and 0 <= pages[seq[t], pos[t] // page] < npages:
                    for h in range(heads):
                        ref[t, h] = R.chunk_values(want[pages[seq[t], pos[t] // page], h], kind, page, dim)[pos[t] % page]
            exact = torch.from_numpy(ref.reshape(ntok, -1)).float().to(dtype(out))  # binary32 holds every value
            assert torch.equal(torch.nan_to_num(got.cpu(), nan=123.0), torch.nan_to_num(exact, nan=123.0)), f"{kind} {out}"


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kinds", PAIRS)
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_write_read(dim, kinds, name):
    """Ragged sequences, each format, width and type; pages that end inside a sequence's new tokens."""
    print(f"kv write {dim} {kinds} {name}", flush=True)
    rng = np.random.default_rng(dim)
    lens, new = [1, 16, 17, 40, 5, 100], [1, 16, 3, 33, 0, 20]
    off = np.concatenate([[0], np.cumsum(new)])
    x = (rng.standard_normal((off[-1], 3 * dim)) * np.exp(rng.standard_normal(3 * dim))).astype(np.float32)
    check(kinds, x, lens, off, 16, dim, 3, name)


@pytest.mark.parametrize("page", [16, 48, 64, 4096])
@pytest.mark.parametrize("heads", [1, 5])
def test_decode_rows(page, heads):
    """One token a sequence without offsets, lengths at the ends of pages; pages past the end of the table
    hold anything."""
    rng = np.random.default_rng(page)
    lens = [1, page - 1, page, page + 1, 2 * page, 2 * page + 7, 3]
    x = rng.standard_normal((len(lens), heads * 64)).astype(np.float32)
    check(("q8_0", "iq4_nl"), x, lens, None, page, 64, heads, missing=0x7FFFFFFF)


def test_positions_that_do_not_exist():
    """Lengths of zero and below the new tokens, past the table, missing pages, tokens of no sequence."""
    rng = np.random.default_rng(5)
    lens = [0, 2, 100, 40, -7, 33]
    off = np.array([2, 3, 8, 12, 20, 21, 30])
    pages, npages = R.tables(rng, lens, 16, width=3)
    pages[3, 1], pages[5, 2] = -1, npages  # the middle of one, the end of another
    x = rng.standard_normal((35, 128)).astype(np.float32)
    for kinds in PAIRS:
        check(kinds, x, lens, off, 16, 64, 2, pages=pages, npages=npages)


def test_offsets_out_of_range():
    """Offsets past the tokens are clamped."""
    rng = np.random.default_rng(6)
    lens, off = [20, 30, 40], np.array([-5, 3, 9, 1000])
    x = rng.standard_normal((16, 64)).astype(np.float32)
    check(("q8_0", "q8_0"), x, lens, off, 16, 64, 1)


def test_blocks_out_of_the_ordinary():
    """Zeros, one value, equal magnitudes of both signs, ties of the rounding and between levels, scales that
    underflow or overflow binary16, infinities and NaN beside finite blocks."""
    rng = np.random.default_rng(7)
    x = np.zeros((14, 64), np.float32)
    x[1, 5] = -3.0
    x[2] = np.where(np.arange(64) % 2, 1.5, -1.5)
    x[3] = np.where(np.arange(64) % 3, 2.5, -2.5)
    x[4, :32] = np.arange(32) + 0.5
    x[4, 0] = 127.0
    x[5, :] = np.resize((R.LEVELS[:-1] + R.LEVELS[1:]) / 2, 64)
    x[5, 0], x[5, 32] = -127.0, 127.0
    x[6] = rng.standard_normal(64) * 1e-9
    x[7] = rng.standard_normal(64) * 1e-41
    x[8] = rng.standard_normal(64) * 1e30
    x[9] = rng.standard_normal(64) * 60000
    x[10, :32], x[10, 32:] = rng.standard_normal(32), -rng.standard_normal(32)
    x[11] = 2.0 ** -149
    x[12] = -0.0
    x[13] = rng.uniform(-1, 1, 64)
    for kinds in PAIRS:
        check(kinds, x, [14], [0, 14], 16, 64, 1)
    for odd in (np.inf, -np.inf, np.nan):
        y = rng.standard_normal((3, 64)).astype(np.float32)
        want = {k: R.stored(y, k) for k in R.FORMATS}
        z = y.copy()
        z[1, 7] = odd
        for kind in R.FORMATS:
            cache = M.KvCache.empty(R.FORMATS[kind], R.FORMATS[kind], 1, 1, 64, 16)
            args = dev(np.zeros((1, 1), np.int32)), dev(np.array([3], np.int32))
            M.qmm_kv_write(cache, *args, dev(z), seg_off=dev(np.array([0, 3], np.int32)))
            got = host(M.qmm_kv_read(cache, *args, k=dtype("f32"), seg_off=dev(np.array([0, 3], np.int32)), ntok=3)[0])
            keep = np.ones((3, 64), bool)
            keep[1, :32] = False
            assert np.array_equal(got[keep], want[kind][keep].astype(np.float32)), kind
            if kind == "f16":
                assert np.array_equal(got, z.astype(np.float16).astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("pad,offset", [(3, 0), (0, 1), (16, 8), (5, 3)])
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_strides(pad, offset, name):
    """Rows at any stride and start; what lies between the rows read stays; a cache of pages that hold keys and
    values together."""
    import torch
    rng = np.random.default_rng(pad)
    ntok, heads, dim, page = 21, 3, 96, 16
    width = heads * dim
    ld = width + pad
    row = 34 * dim // 32
    both = torch.full((4, 2, heads, page, row), 0xA5, dtype=torch.uint8, device="cuda")
    cache = M.KvCache(M.QMM_Q8_0, M.QMM_Q8_0, both[:, 0], both[:, 1])
    pages = np.array([[3, 1, -1]], np.int32)
    args = dev(pages)[:, :2], dev(np.array([ntok], np.int32))
    off = dev(np.array([0, ntok], np.int32))
    x = rng.standard_normal((2, ntok, width)).astype(np.float32)
    views = []
    for i in range(4):
        store = torch.full((offset + ntok * ld,), 7.0, dtype=dtype(name), device="cuda")
        views.append(store[offset:].view(ntok, ld)[:, :width])
    for i in range(2):
        views[i].copy_(dev(x[i]))
    M.qmm_kv_write(cache, *args, views[0], views[1], seg_off=off)
    k, v = M.qmm_kv_read(cache, *args, k=views[2], v=views[3], seg_off=off)
    for i in range(2):
        want = torch.from_numpy(R.stored(host(views[i].float()).reshape(ntok, heads, dim), "q8_0")).float().to(dtype(name))
        assert torch.equal((k, v)[i].cpu(), want.view(ntok, width))
        if pad:
            gap = views[2 + i].as_strided((ntok - 1, pad), (ld, 1), views[2 + i].storage_offset() + width)
            assert (gap == 7.0).all()
    assert (both[0] == 0xA5).all() and (both[2] == 0xA5).all()


def test_one_side_alone():
    """Keys without values and the other way round."""
    import torch
    rng = np.random.default_rng(9)
    x = dev(rng.standard_normal((2, 128)).astype(np.float32))
    pages, lens = dev(np.array([[0], [1]], np.int32)), dev(np.array([4, 16], np.int32))
    cache = M.KvCache.empty(M.QMM_Q8_0, M.QMM_F16, 2, 1, 128, 16)
    M.qmm_kv_write(cache, pages, lens, k=x)
    assert (cache.v == 0).all() and (cache.k != 0).any()
    k0 = cache.k.clone()
    M.qmm_kv_write(cache, pages, lens, v=x)
    assert torch.equal(cache.k, k0)
    k, v = M.qmm_kv_read(cache, pages, lens, v=torch.float16)
    assert k is None and torch.equal(v, x.half())


def test_far_pages():
    """Pages past 4 GiB of the cache."""
    rng = np.random.default_rng(11)
    npages, heads, page, dim = 70000, 4, 64, 256
    cache = M.KvCache.empty(M.QMM_F16, M.QMM_Q8_0, npages, heads, dim, page)
    pages = np.array([[npages - 1, 3, npages // 2]], np.int32)
    x = rng.standard_normal((150, heads * dim)).astype(np.float32)
    args = dev(pages), dev(np.array([150], np.int32))
    off = dev(np.array([0, 150], np.int32))
    M.qmm_kv_write(cache, *args, dev(x), dev(x), seg_off=off)
    k, v = M.qmm_kv_read(cache, *args, k=dtype("f32"), v=dtype("f32"), seg_off=off, ntok=150)
    assert np.array_equal(host(k), R.stored(x, "f16").astype(np.float32))
    assert np.array_equal(host(v), R.stored(x, "q8_0").astype(np.float32))


def test_many_sequences():
    """Thousands of sequences, empty ones among them, one token to a few each."""
    rng = np.random.default_rng(12)
    nseq, page, dim = 3001, 16, 64
    new = rng.integers(0, 3, nseq)
    lens = (new + rng.integers(0, 20, nseq)).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    pages, npages = R.tables(rng, lens, page)
    x = rng.standard_normal((off[-1], dim)).astype(np.float32)
    cache = M.KvCache.empty(M.QMM_IQ4_NL, M.QMM_Q8_0, npages, 1, dim, page)
    args = dev(pages), dev(lens)
    M.qmm_kv_write(cache, *args, dev(x), dev(x), seg_off=dev(off))
    k, v = M.qmm_kv_read(cache, *args, k=dtype("f32"), v=dtype("f32"), seg_off=dev(off), ntok=int(off[-1]))
    assert np.array_equal(host(k), R.stored(x, "iq4_nl").astype(np.float32))
    assert np.array_equal(host(v), R.stored(x, "q8_0").astype(np.float32))


def test_streams_and_graphs():
    """A call on a stream given by handle, and writes with reads behind them in a captured graph whose rows, lengths and
    pages change between the replays, eager calls of another cache beside them."""
    import torch
    rng = np.random.default_rng(8)
    lens = np.array([40, 7, 100], np.int32)
    off = dev(np.array([0, 5, 6, 26], np.int32))
    pages, npages = R.tables(rng, lens, 16, width=9)
    pages, lens = dev(pages), dev(lens)
    caches = [M.KvCache.empty(M.QMM_Q8_0, M.QMM_IQ4_NL, npages, 2, 64, 16) for _ in range(2)]
    x = dev(rng.standard_normal((26, 128)).astype(np.float32))
    outs = [[torch.empty_like(x) for _ in range(2)] for _ in range(2)]

    def run(i, stream=None):
        M.qmm_kv_write(caches[i], pages, lens, x, x, seg_off=off, stream=stream)
        M.qmm_kv_read(caches[i], pages, lens, k=outs[i][0], v=outs[i][1], seg_off=off, stream=stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(0)
    run(1, side.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and torch.equal(caches[0].k, caches[1].k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(0)
    for step in range(4):
        x.normal_()
        lens.copy_(dev(np.array([40 - step, 7 + 3 * step, 100 - 20 * step], np.int32)))
        pages.copy_(pages.roll(step, 1))
        g.replay()
        run(1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)


def test_many_rows():
    """More rows than workgroups fit at once, so that the keys and values of a row are one workgroup's."""
    rng = np.random.default_rng(9)
    new = [1500, 1, 700, 0, 900]
    off = np.concatenate([[0], np.cumsum(new)])
    x = (rng.standard_normal((off[-1], 6 * 64)) * np.exp(rng.standard_normal(6 * 64))).astype(np.float32)
    check(("q8_0", "iq4_nl"), x, [1600, 1, 705, 3, 900], off, 64, 64, 6)
