"""Sizes at the ends of the ranges that the norm, routing, dispatch and value calls take are refused by
status, not by a failed launch.  CPU only, no pointer is followed."""
import ctypes as C

import pytest

import moe_expert_amd as M

FAKE = C.c_void_p(0x100000)


@pytest.mark.parametrize("k,ncols", [(32, (1 << 29) - 1), (32, (1 << 29) - 31), (64, (1 << 28) - 1), (32 * 31, (1 << 29) // 31),
                                     (1 << 30, 16), (32, 1 << 29)])
def test_values_past_one_launch(k, ncols):
    """Eight threads a block in workgroups of 256: the last block counts whose grid stays below 2^32
    threads are 2^29 - 32."""
    assert ncols * (k // 32) > (1 << 29) - 32
    assert M.lib().qmm_dequantize_q8_1(FAKE, k, ncols, M.QMM_TYPE_F32, FAKE, k, None) == -2
