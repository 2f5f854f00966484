"""GPU tests of the attention's split at the sizes where its ways part: 64, 128 and more sequences, tables whose length
on the line is counted in units of many steps, stale entries of a table, offsets that decrease."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import kv_refs as R
from tests.gpu_util import dev, host
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nseq", [64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("longest,width", [(60, 4), (60, 40), (700, 44), (2500, 160)])
def test_sequences(nseq, longest, width):
    """Ragged sequences, empty ones on both sides of the 64th and at the ends, short tables that are not split, short sequences behind
    wide ones, and long ones; one token of each, and up to three."""
    print(f"sequences {nseq} {longest} {width}", flush=True)
    rng = np.random.default_rng(nseq + longest)
    lens = rng.integers(1, longest, nseq)
    lens[rng.integers(0, nseq, 3)] = longest
    for i in (0, 62, 63, 64, 65, 126, 127, 128, nseq - 1):
        if i < nseq and i % 2 == nseq % 2:
            lens[i] = 0
    lens = [int(x) for x in lens]
    Case(lens, kinds=("q8_0", "q8_0"), heads=4, kv=2, dim=64, width=width).check()
    new = [min(n, int(k)) for n, k in zip(lens, rng.integers(0, 4, nseq))]
    Case(lens, new=new, kinds=("f16", "f16"), heads=4, kv=1, dim=64, width=width).check(window=0 if longest < 100 else 90)


@pytest.mark.parametrize("nseq", [17, 90, 140])
def test_units_of_many_steps(nseq):
    """Tables as wide as they may be: the line is counted in units of 2, 8 or 16 steps, whatever the lengths."""
    page, width = 4096, 1 << 18
    rng = np.random.default_rng(nseq)
    lens = [int(x) for x in rng.integers(1, 200, nseq)]
    lens[1], lens[nseq // 2], lens[-1] = 9000, 0, 5000
    c = Case(lens, kinds=("q8_0", "iq4_nl"), heads=2, kv=1, dim=64, page=page)
    want = c.want()
    pages, ln, _ = c.args()
    import torch
    wide = torch.full((nseq, width), -1, dtype=torch.int32, device="cuda")
    wide[:, :pages.shape[1]] = pages
    out, lse = M.qmm_kv_attend(c.q, c.cache(), wide, ln, scale=c.scale, lse=True)
    c.compare(out, lse, want, "f32")


@pytest.mark.parametrize("kinds", [("f16", "f16"), ("f16", "q8_0"), ("q8_0", "q8_0"), ("iq4_nl", "iq4_nl")])
def test_stale_entries(kinds):
    """Entries behind a sequence's pages that name real pages, full of NaN and infinities, and numbers of no page: they
    change no bit.  Lengths at the ends of pages, empty sequences and ones of fewer positions than tokens among them."""
    import torch
    lens, new = [16, 32, 48, 17, 0, 2, 300, 1], [1, 2, 1, 1, 1, 4, 3, 1]
    c = Case(lens, new=new, kinds=kinds, heads=6, kv=2, dim=64, page=16, width=24)
    clean, lse = c.run()
    c.compare(clean, lse, c.want(), "f32")
    used = {int(c.pages[s, i]) for s, n in enumerate(lens) for i in range(-(-n // 16))}
    spare = [p for p in range(c.npages) if p not in used]
    assert spare
    for raw, kind in zip(c.raw, kinds):
        if kind == "f16":
            raw[spare] = np.where(np.arange(64) % 2, np.nan, np.inf)
        else:
            raw.reshape(c.npages, c.kv, -1)[spare, :, 16 * 2 * R.FACTOR[kind]:] = np.tile(np.array([0x00, 0x7C], np.uint8), 16 * 2)
    for fill in (spare[0], spare[-1], c.npages, 0x7FFFFFFF, -5):
        for s, n in enumerate(lens):
            c.pages[s, -(-n // 16):] = fill
        got, lse2 = c.run()
        assert torch.equal(got, clean) and torch.equal(lse, lse2)


@pytest.mark.parametrize("nseq", [6, 100, 130, 2000])
def test_offsets_that_rise_and_fall(nseq):
    """Offsets that give the sequences more tokens than there are: nothing is written, whatever the lengths."""
    ntok = 12
    off = np.where(np.arange(nseq + 1) % 2, ntok, 0).astype(np.int32)
    for longest in (30, 900):
        lens = [longest - i % 7 for i in range(nseq)]
        c = Case(lens[:1], off=[0, ntok], heads=2, kv=1, dim=64, page=64)
        c.lens, c.off = lens, off
        c.pages = np.repeat(c.pages, nseq, axis=0)
        got, lse = c.run()
        assert (host(got) == 7.0).all() and (host(lse) == 7.0).all()


@pytest.mark.parametrize("nseq,ntok,kv", [(16384, 1536, 1), (16384, 4096, 3), (128, 200000, 1)])
def test_offsets_whose_tokens_are_too_many_to_count(nseq, ntok, kv):
    """As many tokens, of as long sequences, that the steps of all of them pass 2^31."""
    import torch
    cache = M.KvCache.empty(M.QMM_F16, M.QMM_F16, 1, kv, 64, 4096)
    pages = torch.zeros(nseq, 64, dtype=torch.int32, device="cuda")
    lens = torch.full((nseq,), 64 * 4096, dtype=torch.int32, device="cuda")
    off = dev(np.where(np.arange(nseq + 1) % 2, ntok, 0).astype(np.int32))
    q = torch.ones(ntok, kv * 64, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((ntok, kv), 7.0, device="cuda")
    M.qmm_kv_attend(q, cache, pages, lens, seg_off=off, out=out, lse=lse)
    assert (out == 7.0).all() and (lse == 7.0).all()


def test_offsets_that_fall():
    """Every sequence without a token, by offsets that only fall: nothing is written."""
    c = Case([40] * 300, off=np.arange(300, -1, -1).astype(np.int32).clip(2), heads=2, kv=1, dim=64)
    got, lse = c.run()
    assert (host(got) == 7.0).all() and (host(lse) == 7.0).all()
