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


def round24(x, drop):
    """Integers over 2^drop rounded to nearest even, to 24 bits: x in [2^(23 + drop), 2^(24 + drop))."""
    half, low = np.int64(1) << (drop - 1), x & ((np.int64(1) << drop) - 1)
    up = (low > half) | ((low == half) & (x >> drop & 1 == 1))
    return (x >> drop) + up


def test_quotient_by_127():
    """The write kernel's amax / 127, a product with 1 / 127 and one residual step in binary32 (qmm_kv.hip), is the
    correctly rounded quotient of every significand: in integers, each rounding by itself.  (Every exponent gives the
    same, as long as nothing is subnormal; the kernel takes it for quotients from 2^-100 on.)"""
    per = np.float32(1) / np.float32(127)  # P 2^-30
    P = np.int64(float(per) * 2.0 ** 30)
    assert float(P) == float(per) * 2.0 ** 30 and 1 << 23 <= P < 1 << 24
    v = np.arange(1 << 23, 1 << 24, dtype=np.int64)
    # 2^23 / 127 = 66052: quotients have 17 or 18 bits before the point, so 24 significant bits end at 2^-7 or 2^-6
    exact = v * P  # of 2^-30
    small = exact < np.int64(1) << 47  # below 2^17
    near = np.where(small, round24(exact, 23), round24(exact, 24) << 1)  # of 2^-7
    rest = (v << 7) - 127 * near  # of 2^-7; exact in binary32, of at most 24 bits
    assert (np.abs(rest) < 1 << 24).all()
    total = (near << 30) + rest * P  # of 2^-37
    small = total < np.int64(1) << 54
    got = np.where(small, round24(total, 30), round24(total, 31) << 1)
    step = np.where(v < 127 << 17, 1, 2)  # v / 127 below 2^17: of 2^-7
    off = np.abs(127 * got - (v << 7))
    assert (2 * off <= 127 * step).all()  # no nearer number of 24 bits; 127 step is odd or twice odd: a tie would be equal
    tie = 2 * off == 127 * step
    assert not tie.any() or (got[tie] // step[tie] % 2 == 0).all()
