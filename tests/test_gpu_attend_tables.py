"""GPU tests of the attention's split: offsets that decrease."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests.gpu_util import dev, host
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu


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
