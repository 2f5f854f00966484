"""More refusals of the key-value cache's calls, and the reading of its arguments.  CPU only, no pointer is followed."""
import ctypes as C

import numpy as np

import moe_expert_amd as M
from tests.test_kv_cpu import ATTEND, FAKE, cache, struct
from tests.test_operators_cpu import Fake, refused


def test_attend_in_place():
    """out is not q: by status, and in the binding whatever q's rows are."""
    import torch
    c = struct()
    a = dict(ATTEND, cache=C.addressof(c), q=FAKE, out=FAKE)
    assert M.lib().qmm_kv_attend(*a.values()) == -1
    f32, i32 = torch.float32, torch.int32
    q = Fake((7, 256), f32)
    refused(M.qmm_kv_attend, q, cache(), Fake((3, 4), i32), Fake((3,), i32), seg_off=Fake((4,), i32), out=q, ws=Fake((1 << 24,), torch.uint8))
