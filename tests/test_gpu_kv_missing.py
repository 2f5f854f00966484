"""GPU test of what a read gives for positions that do not exist: zeros to the bit."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import kv_refs as R
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", ["f16", "q8_0", "iq4_nl"])
def test_missing_positions_are_positive_zeros(dim, kind):
    """Empty sequences, lengths below the new tokens, missing pages, a length past the table, beside rows that exist and whose
    blocks of zeros keep the format's zeros; few rows and many."""
    import torch
    heads, page = 2, 16
    for copies in (1, 200):
        lens = [0, 3, 40, 20, -2] * copies
        new = [2, 5, 3, 4, 1] * copies
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pages, npages = R.tables(np.random.default_rng(dim), lens, page, width=2)
        pages[3::5, 1] = npages
        cache = M.KvCache.empty(R.FORMATS[kind], R.FORMATS[kind], npages, heads, dim, page)
        seq, pos = R.positions(off, lens, int(off[-1]), len(lens))
        there = np.array([0 <= p < 2 * page and 0 <= pages[s, p // page] < npages for s, p in zip(seq, pos)])
        assert there.any() and not there.all()
        for out, bits in ((torch.float32, np.uint32), (torch.float16, np.uint16), (torch.bfloat16, np.uint16)):
            k = torch.full((int(off[-1]), heads * dim), 7.0, dtype=out, device="cuda")
            v = torch.full_like(k, 7.0)
            M.qmm_kv_read(cache, dev(pages), dev(np.asarray(lens, np.int32)), k=k, v=v, seg_off=dev(off))
            for t in (k, v):
                assert (host(t.view(torch.int16 if bits == np.uint16 else torch.int32)).view(bits)[~there] == 0).all()
                assert (host(t.float())[there] == 0).all()
