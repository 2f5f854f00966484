"""GPU tests of the attention over the paged key-value cache (qmm_kv_attend) against its definition in 64 bits,
within the bound that its arithmetic gives."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import kv_refs as R
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

PAIRS = [("f16", "f16"), ("f16", "q8_0"), ("f16", "iq4_nl"), ("q8_0", "q8_0"), ("q8_0", "iq4_nl"), ("iq4_nl", "iq4_nl")]


def dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


class Case:
    """A random cache with its values, tables and queries."""

    def __init__(self, lens, new=None, kinds=("q8_0", "q8_0"), dim=128, heads=4, kv=2, page=16, name="f32", seed=1, extra=0, width=None,
                 qscale=1.0, kscale=1.0, off=None):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.kinds, self.page, self.heads, self.kv, self.dim, self.name = rng, lens, kinds, page, heads, kv, dim, name
        self.off = off if off is not None else None if new is None else np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.pages, self.npages = R.tables(rng, lens, page, width=width)
        self.raw, self.val = [], []
        for kind, scale in zip(kinds, (kscale, 1.0)):
            raw, val = R.random_cache(rng, kind, self.npages, kv, page, dim, scale)
            self.raw.append(raw)
            self.val.append(val)
        self.ntok = (len(lens) if self.off is None else int(max(self.off))) + extra
        x = (qscale * rng.standard_normal((self.ntok, heads * dim))).astype(np.float32)
        self.q = dev(x).to(dtype(name))
        self.scale = dim ** -0.5

    def cache(self):
        return M.KvCache(R.FORMATS[self.kinds[0]], R.FORMATS[self.kinds[1]], dev(self.raw[0]), dev(self.raw[1]))

    def args(self):
        return (dev(self.pages), dev(np.asarray(self.lens, np.int32)), None if self.off is None else dev(np.asarray(self.off, np.int32)))

    def want(self, window=0, q=None):
        q = host((self.q if q is None else q).float())
        return R.attend(q, *self.val, self.pages, self.lens, self.off, self.page, self.heads, self.scale, window)

    def compare(self, got, lse, want, out):
        o, l, bound, lbound, live = want
        rel, tiny = R.HALF_ULP[out]
        got, lse = host(got.float()).astype(np.float64), host(lse).astype(np.float64)
        err = np.abs(got - o)[live]
        most = (bound + (np.abs(o) + bound) * rel + tiny)[live]
        print(f"  worst {np.max(err / most, initial=0):.3f} of the bound", flush=True)
        assert (err <= most).all(), f"{(err > most).sum()} outside, worst {np.nanmax(err / most)}, {np.isnan(err).sum()} NaN"
        none = np.isneginf(l) & live[:, None]
        assert np.array_equal(np.isneginf(lse) & live[:, None], none)
        assert (got.reshape(self.ntok, self.heads, -1)[none] == 0).all()
        fin = np.isfinite(l) & live[:, None]
        lerr = np.abs(lse - l)[fin]
        assert (lerr <= lbound[fin]).all(), f"lse: worst {np.nanmax(lerr / lbound[fin])}"
        assert (got[~live] == 7.0).all() and (lse[~live] == 7.0).all()

    def run(self, window=0, out=None, **kw):
        import torch
        out = out or self.name
        o = torch.full((self.ntok, self.heads * self.dim), 7.0, dtype=dtype(out), device="cuda")
        lse = torch.full((self.ntok, self.heads), 7.0, device="cuda")
        pages, lens, off = self.args()
        cache = kw.pop("cache", None) or self.cache()
        return M.qmm_kv_attend(kw.pop("q", self.q), cache, pages, lens, seg_off=off, scale=self.scale, window=window, out=o, lse=lse, **kw)

    def check(self, window=0, out=None):
        got, lse = self.run(window, out)
        self.compare(got, lse, self.want(window), out or self.name)


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kinds", PAIRS)
def test_formats(dim, kinds):
    """Each width and pair of formats, lengths around the tiles' and pages' ends."""
    print(f"attend {dim} {kinds}", flush=True)
    Case([1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300], kinds=kinds, dim=dim, heads=10, kv=2, seed=dim).check()


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kinds", PAIRS)
def test_formats_in_pieces(dim, kinds):
    """The same behind tables wide enough that sequences may be split, and on both sides of that."""
    print(f"attend in pieces {dim} {kinds}", flush=True)
    Case([1, 33, 130, 300, 512, 515, 639], kinds=kinds, dim=dim, heads=10, kv=2, seed=dim, width=40).check()
    for width in (16, 18, 34, 36):
        Case([16 * width, 16 * width - 15, 3], kinds=kinds, dim=dim, heads=10, kv=2, seed=width, width=width).check()


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kinds", [("f16", "f16"), ("q8_0", "iq4_nl")])
def test_types(name, out, kinds):
    print(f"attend {name} -> {out} {kinds}", flush=True)
    Case([5, 77, 200], kinds=kinds, name=name, heads=6, kv=2, dim=64, page=32).check(out=out)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (5, 1), (16, 1), (17, 1), (40, 1), (128, 2), (64, 64)])
@pytest.mark.parametrize("new", [1, 3])
def test_heads(heads, kv, new):
    """Queries a head of keys from one to 64, rows that do not fill a tile of 16 or 32."""
    print(f"attend heads {heads} {kv} new {new}", flush=True)
    Case([40, 3, 90], new=[new] * 3, kinds=("q8_0", "q8_0"), heads=heads, kv=kv, dim=64, page=16).check()


@pytest.mark.parametrize("page", [16, 48, 64, 256, 4096])
@pytest.mark.parametrize("kinds", [("f16", "f16"), ("iq4_nl", "iq4_nl")])
def test_pages(page, kinds):
    print(f"attend page {page} {kinds}", flush=True)
    Case([1, 100, page - 1, page, page + 1], kinds=kinds, page=page, dim=64, heads=2, kv=1).check()


@pytest.mark.parametrize("kinds", PAIRS)
@pytest.mark.parametrize("window", [0, 1, 7, 33, 1000])
def test_new_tokens_and_windows(kinds, window):
    """Ragged new tokens behind cached ones, none in some sequences, more than the sequence holds in one, tokens of
    no sequence before and behind."""
    print(f"attend new {kinds} window {window}", flush=True)
    off = np.cumsum([2, 1, 8, 0, 5, 7, 3]).astype(np.int32)
    Case([90, 8, 50, 200, 4, 33], kinds=kinds, off=off, extra=3, heads=10, kv=2, dim=96, page=16).check(window)


def test_prompt():
    """Hundreds of new tokens of a sequence at once."""
    Case([300, 40], new=[260, 40], heads=6, kv=2, dim=64, page=32).check()
    Case([150], new=[150], heads=3, kv=1, dim=128, page=16, kinds=("f16", "f16")).check(window=20)


def test_empty_rows():
    """Empty sequences, lengths below zero and past the table, pages that are missing: a whole sequence's, its
    first, one in the middle."""
    c = Case([0, -3, 70, 70, 70, 200, 16], new=[1, 2, 2, 3, 2, 4, 1], heads=4, kv=2, dim=64, page=16, width=6)
    c.pages[2, :] = -1
    c.pages[3, 0] = c.npages
    c.pages[4, 2] = -2147483648
    c.check()
    c.check(window=30)


@pytest.mark.parametrize("kinds", PAIRS)
def test_not_a_number_in_unseen_places(kinds):
    """Every place that no row sees holds NaN and infinities, the positions that only later tokens of the
    sequence see among them: they change no bit."""
    c = Case([45, 20, 64, 7], new=[4, 1, 8, 2], kinds=kinds, heads=6, kv=2, dim=64, page=16)
    clean, lse = c.run()
    seen = np.zeros((c.npages, c.page), bool)
    for s, n in enumerate(c.lens):
        for j in range(n):
            seen[c.pages[s, j // 16], j % 16] = True
    for raw, kind in zip(c.raw, kinds):
        if kind == "f16":
            raw[~seen[:, None, :].repeat(c.kv, 1)] = np.nan
        else:
            per = R.FACTOR[kind] * 2
            scales = raw.reshape(c.npages, c.kv, -1)[:, :, 16 * per:].reshape(c.npages, c.kv, 16, 4).view(np.float16)
            scales[~seen[:, None, :].repeat(c.kv, 1)] = np.nan
    got, lse2 = c.run()
    import torch
    assert torch.equal(got, clean) and torch.equal(lse, lse2)
    # the last token of the first and third sequence holds odd keys and values: only its own rows may show it
    for value in (np.nan, np.inf, -np.inf):
        for s in (0, 2):
            j = c.lens[s] - 1
            for raw, kind in zip(c.raw, kinds):
                chunk = raw[c.pages[s, j // 16]]
                if kind == "f16":
                    chunk[:, j % 16, 5] = value
                else:
                    per = R.FACTOR[kind] * 2
                    chunk.reshape(c.kv, -1)[:, 16 * per:].reshape(c.kv, 16, 4).view(np.float16)[:, j % 16, 1] = value
        got, lse2 = c.run()
        last = [int(c.off[1]) - 1, int(c.off[3]) - 1]
        keep = [t for t in range(c.ntok) if t not in last]
        assert torch.equal(got[keep], clean[keep]) and torch.equal(lse[keep], lse2[keep])
        for t in last:
            assert not torch.isfinite(got[t]).all()


def test_queries_that_are_not_finite():
    """A row of q with NaN or an infinity gives NaN in its own outputs alone."""
    c = Case([30, 50], new=[2, 3], heads=6, kv=2, dim=64, page=16)
    clean, _ = c.run()
    q = c.q.clone()
    q[1, 64 * 3 + 5], q[4, 2] = float("nan"), float("inf")
    got, _ = c.run(q=q)
    g, w = host(got).reshape(5, 6, 64), host(clean).reshape(5, 6, 64)
    odd = np.zeros((5, 6), bool)
    odd[1, 3] = odd[4, 0] = True
    assert np.array_equal(g[~odd], w[~odd]) and np.isnan(g[odd]).all()


@pytest.mark.parametrize("kinds", [("f16", "f16"), ("q8_0", "q8_0"), ("iq4_nl", "iq4_nl")])
@pytest.mark.parametrize("qscale,kscale", [(1e-6, 1.0), (12.0, 1.0), (1e-3, 1e3), (30000.0, 1e-3), (1e8, 1e-4), (0.0, 1.0)])
def test_scores_of_all_sizes(kinds, qscale, kscale):
    """Scores near zero, peaked ones, small and large queries."""
    print(f"attend scores {kinds} {qscale} {kscale}", flush=True)
    Case([400, 17], kinds=kinds, heads=4, kv=2, dim=128, page=16, qscale=qscale, kscale=kscale).check()


def test_scale_of_any_sign():
    c = Case([100], heads=2, kv=1, dim=64)
    for scale in (0.0, -0.3, 2.0):
        c.scale = scale
        c.check()


@pytest.mark.parametrize("kinds", [("f16", "f16"), ("f16", "q8_0")])
def test_one_large_score_and_many_small(kinds):
    """A first position whose score is far above the others', whose weights together still count, in a
    long cache: they are not lost in the products' narrower parts."""
    n = 20000
    c = Case([n], kinds=kinds, heads=2, kv=1, dim=64, page=64, kscale=0.01)
    q = host(c.q)[0].reshape(2, 64)
    for top in (9.0, 14.0, 18.0):
        k = (q.mean(axis=0) / np.square(q.mean(axis=0)).sum()) / c.scale * top
        c.raw[0][c.pages[0, 0], 0, 0] = k.astype(np.float16)
        c.val[0][c.pages[0, 0], 0, 0] = k.astype(np.float16)
        # values whose mean is far from zero, but at the first position
        if kinds[1] == "f16":
            c.raw[1][:] = np.abs(c.raw[1]) + 1
            c.raw[1][c.pages[0, 0], 0, 0] = 0
            c.val[1] = c.raw[1].astype(np.float64)
        c.check()


def test_long():
    """Lengths that need every split, ragged beside short ones."""
    print("attend long", flush=True)
    Case([70001, 5, 3000, 1], kinds=("q8_0", "iq4_nl"), heads=5, kv=1, dim=64, page=128).check()


def test_many_sequences():
    """More sequences than a workgroup scans at once, most of one or no token."""
    rng = np.random.default_rng(2)
    new = rng.integers(0, 3, 1500)
    lens = [int(x) for x in new + rng.integers(0, 30, 1500)]
    Case(lens, new=new, heads=2, kv=1, dim=64, kinds=("f16", "f16")).check()


@pytest.mark.parametrize("lens,kv", [([40000], 8), ([50000], 7), ([9000, 30000, 7, 0, 2000], 5), ([12000] * 3, 8), ([3000, 0, 70] * 20, 6)])
@pytest.mark.parametrize("kinds", [("f16", "q8_0"), ("iq4_nl", "iq4_nl")])
def test_long_lines(lens, kv, kinds):
    """Enough steps that workgroups take unequal lengths in turn, of one sequence and of several, whose ends lie in either."""
    print(f"attend {lens[:5]} {kv} {kinds}", flush=True)
    Case(lens, kinds=kinds, heads=kv, kv=kv, dim=64, page=64, seed=kv).check()


def test_long_line_of_many_sequences():
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 900, 300)]
    Case(lens, kinds=("q8_0", "q8_0"), heads=4, kv=2, dim=64, page=32).check()


def test_workspace_too_small():
    import torch
    c = Case([400, 90], heads=4, kv=2, dim=64)
    need = M.qmm_kv_attend_workspace(c.cache(), 2, 4, 2, c.pages.shape[1])
    for n in (16, need - 1):
        with pytest.raises(ValueError, match="ws must be"):
            c.run(ws=torch.empty(n, dtype=torch.uint8, device="cuda"))
    c.compare(*c.run(ws=torch.empty(need, dtype=torch.uint8, device="cuda")), c.want(), "f32")


def test_offsets_that_decrease():
    """More tokens than there are, by offsets that do not stand for any split: nothing is written."""
    off = np.array([0, 4, 2, 6], np.int32)
    c = Case([40, 50, 60], off=off, heads=2, kv=1, dim=64)
    got, lse = c.run()
    assert (host(got) == 7.0).all() and (host(lse) == 7.0).all()
    c = Case([40] * 300, off=np.arange(300, -1, -1).astype(np.int32).clip(2), heads=2, kv=1, dim=64)
    got, lse = c.run()
    assert np.isfinite(host(got)).all()


@pytest.mark.parametrize("pad,offset", [(3, 0), (0, 1), (16, 8), (5, 3)])
@pytest.mark.parametrize("name", ["f32", "f16"])
def test_strides(pad, offset, name):
    """Rows of q and out at any stride and start, tables that are views, pages that hold keys and values
    together; what lies between the rows stays."""
    import torch
    c = Case([40, 90], new=[3, 2], kinds=("q8_0", "q8_0"), heads=6, kv=3, dim=96, page=16, name=name)
    width, ld = 6 * 96, 6 * 96 + pad
    views = []
    for _ in range(2):
        store = torch.full((offset + c.ntok * ld,), 7.0, dtype=dtype(name), device="cuda")
        views.append(store[offset:].view(c.ntok, ld)[:, :width])
    views[0].copy_(c.q)
    both = torch.stack([dev(c.raw[0]), dev(c.raw[1])], dim=1)
    cache = M.KvCache(M.QMM_Q8_0, M.QMM_Q8_0, both[:, 0], both[:, 1])
    pages, lens, off = c.args()
    wide = torch.full((2, pages.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, :pages.shape[1]] = pages
    got, lse = M.qmm_kv_attend(views[0], cache, wide[:, :pages.shape[1]], lens, seg_off=off, scale=c.scale, out=views[1], lse=True)
    c.compare(got, lse, c.want(), name)
    if pad:
        gap = views[1].as_strided((c.ntok - 1, pad), (ld, 1), views[1].storage_offset() + width)
        assert (gap == 7.0).all()


def test_far_pages():
    """A cache of more than 4 GiB a side, pages at its end."""
    npages, heads, page, dim = 70000, 4, 64, 256
    rng = np.random.default_rng(3)
    cache = M.KvCache.empty(M.QMM_F16, M.QMM_F16, npages, heads, dim, page)
    pages = np.array([[npages - 1, 5, npages // 2 + 7]], np.int32)
    x = rng.standard_normal((2, 150, heads * dim)).astype(np.float32)
    off = dev(np.array([0, 150], np.int32))
    lens = dev(np.array([150], np.int32))
    M.qmm_kv_write(cache, dev(pages), lens, dev(x[0]), dev(x[1]), seg_off=off)
    c = Case([150], kinds=("f16", "f16"), heads=heads, kv=heads, dim=dim, page=page)
    c.pages = np.array([[0, 1, 2]], np.int32)
    for i in range(2):
        v = np.zeros((3 * page, heads, dim))
        v[:150] = x[i].astype(np.float16).reshape(150, heads, dim)
        c.val[i] = v.reshape(3, page, heads, dim).transpose(0, 2, 1, 3)
    want = c.want()
    got, lse = M.qmm_kv_attend(c.q, cache, dev(pages), lens, lse=True)
    c.compare(got, lse, want, "f32")


def test_same_bits_again():
    """Two calls in a row, and a batch's row beside other rows' lengths, give the same bits."""
    import torch
    c = Case([5000, 17, 900, 64], heads=10, kv=2, dim=128, page=64)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_joined_by_lse():
    """Two halves of a cache joined by their lse give the whole's attention."""
    import torch
    c = Case([256], heads=4, kv=2, dim=64, page=16)
    pages, lens, _ = c.args()
    cache = c.cache()
    half = [M.qmm_kv_attend(c.q, cache, p.contiguous(), torch.full_like(lens, 128), scale=c.scale, lse=True)
            for p in (pages[:, :8], pages[:, 8:])]
    whole, lse = M.qmm_kv_attend(c.q, cache, pages, lens, scale=c.scale, lse=True)
    l = torch.stack([h[1] for h in half]).double()
    w = torch.softmax(l, dim=0)[..., None]
    joined = (w * torch.stack([h[0].view(1, 4, 64) for h in half]).double()).sum(dim=0).view(1, -1)
    o, _, bound, lbound, _ = c.want()
    assert (np.abs(host(joined) - o) <= 3 * bound).all()
    assert (np.abs(host(torch.logsumexp(l, dim=0) - lse.double())) <= 3 * lbound).all()


def test_streams_and_graphs():
    """On a side stream given by handle, and in two captured graphs with a workspace each whose lengths change between the
    replays, eager calls beside them."""
    import torch
    c = Case([600, 33, 1000], heads=10, kv=2, dim=128, page=16)
    cache = c.cache()
    pages, lens, _ = c.args()
    side = torch.cuda.Stream()
    want, _ = M.qmm_kv_attend(c.q, cache, pages, lens, scale=c.scale)
    torch.cuda.synchronize()
    got, _ = M.qmm_kv_attend(c.q, cache, pages, lens, scale=c.scale, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)
    graphs = []
    for i in range(2):
        q, now = c.q.clone(), lens.clone()
        need = M.qmm_kv_attend_workspace(cache, 3, 10, 3, pages.shape[1])
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(3, 10, device="cuda")
        M.qmm_kv_attend(q, cache, pages, now, scale=c.scale, out=out, lse=lse, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.qmm_kv_attend(q, cache, pages, now, scale=c.scale, out=out, lse=lse, ws=ws)
        graphs.append((g, q, now, out, lse))
    for step in range(4):
        for i, (g, q, now, out, lse) in enumerate(graphs):
            q.normal_()
            now.copy_(dev(np.array([600 - 17 * step, 33 * i, 1000 // (step + 1)], np.int32)))
        for g, *_ in graphs:
            g.replay()
        ref = [M.qmm_kv_attend(q, cache, pages, now, scale=c.scale, lse=True) for _, q, now, _, _ in graphs]
        torch.cuda.synchronize()
        for (g, q, now, out, lse), (o, l) in zip(graphs, ref):
            assert torch.equal(out, o) and torch.equal(lse, l)


@pytest.mark.parametrize("nseq,longest", [(150, 700), (40, 200), (3, 200)])
def test_graph_of_other_lengths(nseq, longest):
    """Captured calls that plan in a launch of their own, and that do not split: lengths and tables change between the replays."""
    import torch
    rng = np.random.default_rng(nseq)
    c = Case([int(x) for x in rng.integers(0, longest, nseq)], kinds=("q8_0", "iq4_nl"), heads=4, kv=2, dim=64, page=32)
    cache = c.cache()
    pages, lens, _ = c.args()
    out, lse = torch.empty_like(c.q), torch.empty(nseq, 4, device="cuda")
    ws = torch.empty(M.qmm_kv_attend_workspace(cache, nseq, 4, nseq, pages.shape[1]), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        M.qmm_kv_attend(c.q, cache, pages, lens, out=out, lse=lse, ws=ws)
    for step in range(4):
        lens.copy_(lens.roll(1) - step)
        pages.copy_(pages.roll(step, 0))
        ws.fill_(255 * (step % 2))
        g.replay()
        want = M.qmm_kv_attend(c.q, cache, pages, lens, lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_written_then_attended():
    """A request's life: its prompt written and attended, then tokens one and three at a time, against the
    attention over the values as they were stored."""
    import torch
    rng = np.random.default_rng(4)
    heads, kv, dim, page = 6, 2, 64, 16
    cache = M.KvCache.empty(M.QMM_Q8_0, M.QMM_IQ4_NL, 8, kv, dim, page)
    pages = rng.permutation(8)[:6].astype(np.int32)[None]
    x = rng.standard_normal((2, 90, kv * dim)).astype(np.float32)
    val = [np.zeros((8, kv, page, dim)) for _ in range(2)]
    n = 0
    for new in (40, 1, 1, 3, 1, 30, 1):
        rows = slice(n, n + new)
        n += new
        off, lens = dev(np.array([0, new], np.int32)), dev(np.array([n], np.int32))
        M.qmm_kv_write(cache, dev(pages), lens, dev(x[0][rows]), dev(x[1][rows]), seg_off=off)
        for i, kind in enumerate(("q8_0", "iq4_nl")):
            back = R.stored(x[i][rows].reshape(new, kv, dim), kind)
            for t in range(new):
                val[i][pages[0, (n - new + t) // page], :, (n - new + t) % page] = back[t]
        q = dev(rng.standard_normal((new, heads * dim)).astype(np.float32))
        got, lse = M.qmm_kv_attend(q, cache, dev(pages), lens, seg_off=off, lse=True)
        o, l, bound, lbound, _ = R.attend(host(q), *val, pages, [n], [0, new], page, heads, dim ** -0.5, 0)
        assert (np.abs(host(got) - o) <= bound).all() and (np.abs(host(lse) - l) <= lbound).all()
