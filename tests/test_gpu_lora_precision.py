"""GPU tests of qmm_lora's outer product: every inner value enters it in binary32, whatever the size
of the token's other inner values, and infinities of the tables give what the formula gives."""
import numpy as np
import pytest

from tests import operator_refs as R
from tests.test_gpu_lora import inputs, run

pytestmark = pytest.mark.gpu


def reference(x, a, b, ranks, scales, seg_off, adapters, base):
    """(y, bound) in 64 bits.  The bound is that of binary32 sums in any order: an inner sum of k
    products, an outer sum of r, in which an inner value's error passes through its own column of B
    only; the factor and the base's addition."""
    k = x.shape[1]
    y = base.astype(np.float64).copy()
    bound = R.U * np.abs(y)
    for s, i in enumerate(adapters):
        if not 0 <= i < a.shape[0]:
            continue
        t, r, sc = slice(seg_off[s], seg_off[s + 1]), int(ranks[i]), float(scales[i])
        xs, ai, bi = x[t].astype(np.float64), a[i, :r].astype(np.float64), b[i, :, :r].astype(np.float64)
        v = xs @ ai.T
        ev = (k + 1) * R.U * (np.abs(xs) @ np.abs(ai).T)
        y[t] += sc * (v @ bi.T)
        bound[t] += abs(sc) * (ev @ np.abs(bi).T + (r + 3) * R.U * ((np.abs(v) + ev) @ np.abs(bi).T)) + 2 * R.U * np.abs(y[t])
    return y, bound + 2.0 ** -149


@pytest.mark.parametrize("ntok,lens", [(6, [1] * 6), (70, [1, 69]), (1100, [1100])])
@pytest.mark.parametrize("xt", ["f16", "f32"])
def test_small_inner_values_beside_a_large_one(ntok, lens, xt):
    """One rank row is 2^26 times the others, and half of B's rows do not use it: their outputs have
    the bits of their own terms."""
    na = 2
    arrays = list(inputs(31 + ntok, ntok, 320, 100, 16, lens, [i % na for i in range(len(lens))], na, xt, ranks=[16, 11]))
    a, b = arrays[1].astype(np.float64), arrays[2]
    a *= np.sqrt(320)
    a[:, 1:] *= 2.0 ** -13
    a[:, 0] *= 2.0 ** 13
    arrays[1] = a.astype(np.float16)
    assert np.isfinite(arrays[1][:, 0]).all()
    b[:, ::2, 0] = 0
    arrays[7] = np.zeros_like(arrays[7])
    y = run(tuple(arrays))
    want, bound = reference(*arrays)
    err = np.abs(y - want)
    assert (err <= bound).all(), f"{(err > bound).sum()} outside, worst {np.max(err / bound)}"


@pytest.mark.parametrize("ntok", [3, 200, 1100])
def test_infinities_of_the_tables(ntok):
    """An infinite entry of B gives the infinity of the product's sign, and touches nothing else; an
    infinite inner value the same."""
    arrays = list(inputs(5, ntok, 64, 90, 16, [ntok], [0], 1, ranks=[16]))
    clean = run(tuple(arrays))
    x, a, b = arrays[0].astype(np.float64), arrays[1].astype(np.float64), arrays[2]
    v = x @ a[0].T
    sure = np.abs(v) > 1e-3  # the sign of the inner value is beyond doubt
    b[0, 7, 3] = np.inf
    b[0, 60, 12] = -np.inf
    y = run(tuple(arrays))
    sign = np.sign(arrays[4][0])
    for row, j, s in ((7, 3, 1), (60, 12, -1)):
        want = s * sign * np.sign(v[:, j]) * np.inf
        assert np.array_equal(y[sure[:, j], row], want[sure[:, j]])
    keep = [r for r in range(90) if r not in (7, 60)]
    assert np.array_equal(y[:, keep], clean[:, keep])
    arrays = list(inputs(6, ntok, 64, 90, 8, [ntok], [0], 1, ranks=[1]))
    t = ntok // 2
    arrays[0][t, 5] = np.inf
    arrays[1][0, 0, 5] = 0.25
    arrays[2][0, :, 0] = np.where(arrays[2][0, :, 0] == 0, 1, arrays[2][0, :, 0])
    y = run(tuple(arrays))
    assert np.array_equal(y[t], np.sign(arrays[4][0]) * np.sign(arrays[2][0, :, 0].astype(np.float64)) * np.inf)
