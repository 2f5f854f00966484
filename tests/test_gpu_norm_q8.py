"""GPU tests of the norm's q8_1 output in every kernel: unaligned rows and long ones, each input and
output type, in place; the bytes of qmm_quantize_q8_1 on the binary32 norm of an aligned call."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests.test_gpu_norm import TYPES, check, dtype, rows

pytestmark = pytest.mark.gpu


def weights(rng, hidden, offset=0):
    import torch
    return torch.from_numpy((1 + 0.3 * rng.standard_normal(hidden + offset)).astype(np.float32)).cuda()[offset:]


@pytest.mark.parametrize("hidden", [32, 96, 544, 2560, 4064, 4128, 6144, 8192, 8224, 12288, 32768])
@pytest.mark.parametrize("pad,offset", [(3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("name", TYPES)
def test_q8_of_unaligned_rows(hidden, pad, offset, name):
    """Rows read one value at a time: the norm within its bound, and its q8_1 as the quantizer has it."""
    import torch
    print(f"norm q8 {hidden}+{pad} at {offset} {name}", flush=True)
    rng = np.random.default_rng(hidden + pad)
    x, res = rows(rng, 7, hidden, name, pad, offset), rows(rng, 7, hidden, "f32", pad, offset)
    y, res_out = rows(rng, 7, hidden, "f32", pad, offset), rows(rng, 7, hidden, "f32", pad, offset)
    w = weights(rng, hidden, offset)
    yq = torch.full((7, hidden // 32 * 36), 0x5A, dtype=torch.uint8, device="cuda")
    M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=res_out, y=y, yq=yq)
    check(x, res, w, 1e-6, y, yq, res_out, "f32")
    alone = torch.full_like(yq, 0x5A)
    M.qmm_rmsnorm(x, w, 1e-6, res=res, yq=alone)
    assert torch.equal(alone, yq)


@pytest.mark.parametrize("hidden,pad", [(64, 0), (2560, 0), (2560, 1), (9216, 0), (9216, 1)])
@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("yt", TYPES)
def test_q8_beside_each_output_type(hidden, pad, xt, yt):
    """The q8_1 output is of the binary32 norm, not of the rounded output beside it."""
    import torch
    rng = np.random.default_rng(hidden)
    x, w = rows(rng, 5, hidden, xt, pad), weights(rng, hidden)
    y32 = rows(rng, 5, hidden, "f32", pad)
    M.qmm_rmsnorm(x, w, 1e-6, y=y32)
    y = rows(rng, 5, hidden, yt, pad)
    _, yq, _ = M.qmm_rmsnorm(x, w, 1e-6, y=y, yq=True)
    assert torch.equal(y, y32.to(dtype(yt)))
    assert torch.equal(yq, M.qmm_quantize_q8_1(y32.contiguous()))


@pytest.mark.parametrize("ntok,hidden,pad", [(5, 6144, 1), (4, 9216, 0), (4, 9216, 1), (3, 32768, 1), (3, 32767, 0)])
def test_long_rows_in_place(ntok, hidden, pad):
    """The residual updated in place and the norm written over x in rows that are read twice."""
    import torch
    rng = np.random.default_rng(hidden + pad)
    x, res = rows(rng, ntok, hidden, "f32", pad), rows(rng, ntok, hidden, "f32", pad)
    w = weights(rng, hidden)
    q8 = True if hidden % 32 == 0 else None
    want, r = rows(rng, ntok, hidden, "f32", pad), rows(rng, ntok, hidden, "f32", pad)
    _, wantq, _ = M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=r, y=want, yq=q8)
    check(x, res, w, 1e-6, want, wantq, r, "f32")
    _, yq, _ = M.qmm_rmsnorm(x, w, 1e-6, res=res, res_out=res, y=x, yq=q8)
    assert torch.equal(x, want) and torch.equal(res, r)
    assert q8 is None or torch.equal(yq, wantq)
