"""GPU tests of the routing's weights where the bias takes experts out: the softmax is over every expert
whose logit is not -inf or NaN, the bias decides only who can be chosen."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import operator_refs as R
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e,topk,groups", [(24, 4, 1), (128, 8, 1), (256, 8, 8), (320, 6, 4), (1000, 8, 1)])
@pytest.mark.parametrize("renorm", [False, True])
def test_weights_of_a_masking_bias(e, topk, groups, renorm):
    """By hand in 64 bits: the chosen are the best of score + bias among the experts that the bias
    leaves; their weights are shares of the whole softmax, or of their own sum."""
    rng = np.random.default_rng(e)
    z = (2 * rng.standard_normal((50, e))).astype(np.float32)
    z[:, 1] += 6  # a large share lies with experts that the bias takes out
    z[3, 2] = -np.inf
    z[4, 2] = np.nan
    bias = (0.05 * rng.standard_normal(e)).astype(np.float32)
    bias[[1, 5, 11]] = [-np.inf, np.nan, -np.inf]
    ids, w = M.qmm_moe_route(dev(z), topk, bias=dev(bias), ngroups=groups, topk_groups=groups, renorm=renorm)
    ids, w = host(ids), host(w)
    z64 = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    share = np.exp(z64 - z64.max(1, keepdims=True))
    share /= share.sum(1, keepdims=True)
    c = np.where(np.isneginf(z64) | np.isnan(bias), -np.inf, share + bias)
    order = np.argsort(-c, axis=1, kind="stable")[:, :topk + 1]
    gap = np.diff(-np.take_along_axis(c, order, 1)).min(1)
    sure = gap > 8e-7  # binary32 scores and sums decide as these do
    assert sure.mean() > 0.8
    assert np.array_equal(ids[sure], order[sure, :topk])
    want = np.take_along_axis(share, order[:, :topk], 1)
    if renorm:
        want /= want.sum(1, keepdims=True)
    else:
        assert (want.sum(1) < 0.9).any()
    finite = np.where(np.isfinite(z), z, 0)
    spread = (finite.max(1) - finite.min(1))[:, None]
    assert (np.abs(w - want)[sure] <= R.route_weight_bound(want, spread)[sure]).all()
