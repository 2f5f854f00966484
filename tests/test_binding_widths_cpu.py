"""The binding refuses weight vectors of another width than the call's: a longer one is another
model's.  CPU only; buffers for outputs and segment lists may be longer than the call needs."""
import torch

import moe_expert_amd as M
from tests.test_operators_cpu import Fake, refused

F32, F16, I32 = torch.float32, torch.float16, torch.int32


def test_norm_weights():
    x, y = Fake((4, 64), F32), Fake((4, 64), F16)
    refused(M.qmm_rmsnorm, x, Fake((65,), F32), 1e-6, y=y)
    refused(M.qmm_rmsnorm, x, Fake((2, 64), F32), 1e-6, y=y)


def test_routing_bias():
    z = Fake((4, 64), F32)
    refused(M.qmm_moe_route, z, 2, bias=Fake((65,), F32), ids=Fake((4, 2), I32), weights=Fake((4, 2), F32))
    refused(M.qmm_moe_route, z, 2, bias=Fake((128,), F32), ids=Fake((4, 2), I32), weights=Fake((4, 2), F32))


def test_adapter_tables():
    good = dict(x=Fake((4, 64), F16), a=Fake((2, 16, 64), F16), b=Fake((2, 100, 16), F16), ranks=Fake((2,), I32), scales=Fake((2,), F32),
                seg_off=Fake((2,), I32), seg_adapter=Fake((1,), I32), y=Fake((4, 100), F32), base=Fake((4, 100), F32),
                ws=Fake((1 << 20,), torch.uint8))
    for name, bad in (("ranks", Fake((3,), I32)), ("scales", Fake((3,), F32))):
        refused(M.qmm_lora, **dict(good, **{name: bad}))
