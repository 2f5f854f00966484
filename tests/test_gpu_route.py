"""GPU tests of the routing (qmm_moe_route) and the dispatch (qmm_moe_dispatch) against 64-bit
references: ids and lists exactly, weights within their bound."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import operator_refs as R
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu


def dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def run_route(logits, topk, softmax, bias=None, **kw):
    """The call, and the 64-bit reference on the values it read."""
    score = M.QMM_SCORE_SOFTMAX if softmax else M.QMM_SCORE_SIGMOID
    ids, w = M.qmm_moe_route(logits, topk, score=score, bias=None if bias is None else dev(bias), **kw)
    z = host(logits.float())
    return host(ids), host(w), R.route(z, topk, softmax, bias=bias, **kw), z


def check(got_ids, got_w, ref, z, decided=8e-7):
    """ids equal wherever the reference decided by more than the binary32 error of what it compared
    (two sums of two scores below 1, each score within 2 units of 2^-24 and each addition within
    one, and the bias' addition: under 8e-7); weights of those rows within the bound.  Most rows must
    be decided."""
    ids, w, margin = ref
    sure = margin > decided
    assert sure.mean() > 0.75
    assert np.array_equal(got_ids[sure], ids[sure]), f"{(got_ids[sure] != ids[sure]).any(axis=1).sum()} rows differ"
    finite = np.where(np.isfinite(z), z, 0.0)
    spread = (finite.max(axis=1) - finite.min(axis=1))[:, None]
    err = np.abs(got_w[sure] - w[sure])
    assert (err <= R.route_weight_bound(w[sure], spread[sure])).all(), err.max()


CASES = [  # ntok, experts, topk, softmax, bias, groups, kept, group_top, renorm, scale
    (1, 128, 8, True, False, 1, 1, 1, True, 1.0),
    (9, 128, 8, True, False, 1, 1, 1, False, 1.0),
    (700, 128, 8, True, False, 1, 1, 1, True, 1.0),
    (333, 8, 2, True, False, 1, 1, 1, True, 1.0),
    (50, 1, 1, True, False, 1, 1, 1, True, 1.0),
    (65, 5, 5, True, False, 1, 1, 1, False, 2.0),
    (40, 33, 3, False, False, 1, 1, 1, True, 1.0),
    (300, 256, 8, False, True, 8, 4, 2, True, 2.5),
    (90, 160, 6, True, False, 8, 3, 1, False, 16.0),
    (70, 160, 6, True, False, 8, 3, 2, True, 1.0),
    (60, 64, 6, True, True, 1, 1, 1, True, 1.0),
    (60, 63, 7, False, True, 7, 3, 1, True, 1.0),
    (30, 512, 16, False, True, 16, 5, 2, True, 1.0),
    (20, 1024, 64, True, False, 1, 1, 1, True, 1.0),
    (20, 1023, 10, False, True, 1, 1, 1, True, 1.0),
    (12, 1024, 64, False, True, 64, 32, 2, False, 1.0),
    (33, 96, 64, True, False, 1, 1, 1, True, 1.0),
    (25, 64, 4, False, False, 64, 10, 1, True, 1.0),
    (4000, 60, 4, False, False, 1, 1, 1, True, 1.0),
    (15, 300, 20, True, True, 3, 2, 2, True, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
@pytest.mark.parametrize("lt", ["f32", "f16"])
def test_route(case, lt):
    import torch
    n, e, k, softmax, biased, ng, kept, gt, renorm, scale = case
    print(f"route {case} {lt}", flush=True)
    rng = np.random.default_rng(n + e)
    z = (rng.standard_normal((n, e)) * 1.5 + 0.5 * rng.standard_normal(e)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(e)).astype(np.float32) if biased else None
    got = run_route(dev(z).to(dtype(lt)), k, softmax, bias, ngroups=ng, topk_groups=kept, group_top=gt, renorm=renorm, scale=scale)
    check(*got)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("e,k", [(128, 8), (256, 16), (40, 40), (1024, 30)])
def test_route_ties(softmax, e, k):
    """Logits of three values: nearly every choice is a tie, which goes to the lowest expert; runs
    that tie go to the lowest run."""
    rng = np.random.default_rng(e)
    z = rng.integers(0, 3, (60, e)).astype(np.float32)
    z[0] = 1.0
    z[1] = -0.0
    z[1, ::2] = 0.0
    for kw in (dict(), dict(ngroups=4, topk_groups=4, group_top=1), dict(ngroups=4, topk_groups=4, group_top=2)):
        got_ids, got_w, ref, zz = run_route(dev(z), k, softmax, **kw)
        assert np.array_equal(got_ids, ref[0])
        assert (np.abs(got_w - ref[1]) <= R.route_weight_bound(ref[1], 2.0)).all()
    ids, _, ref, _ = run_route(dev(z), min(k, e // 4), softmax, ngroups=4, topk_groups=1)
    assert np.array_equal(ids, ref[0])


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("lt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("e", [24, 128, 320])
def test_route_masked(softmax, lt, e):
    """Masked experts (-inf, NaN), rows with fewer experts than choices, rows with none, rows at the
    type's lowest value, rows with infinities."""
    import torch
    rng = np.random.default_rng(e)
    z = torch.from_numpy(rng.standard_normal((40, e)).astype(np.float32)).to(dtype(lt)).cuda()
    low = torch.finfo(dtype(lt)).min
    z[:, 3] = float("-inf")
    z[0] = float("-inf")
    z[1] = float("nan")
    z[2, 4:] = float("-inf")
    z[3] = low
    z[4] = low
    z[4, 7] = 0.0
    z[5, 11] = float("nan")
    z[6, 9] = float("inf")
    z[7, 9] = float("inf")
    z[7, 12] = float("inf")
    for renorm in (True, False):
        ids, w, ref, zz = run_route(z, 8, softmax, renorm=renorm)
        assert (ids[:2] == -1).all() and (w[:2] == 0).all() and (ids[2, 3:] == -1).all() and (w[2, 3:] == 0).all()
        sure = ref[2] > 1e-6
        assert sure.sum() >= 38
        assert np.array_equal(ids[sure], ref[0][sure])
        assert np.isfinite(w).all()
        assert (np.abs(w - ref[1])[sure] <= R.route_weight_bound(ref[1][sure], 12.0) + 1e-30).all()
    bias = np.zeros(e, np.float32)
    bias[:4] = -np.inf
    bias[5] = np.nan
    ids, w, ref, _ = run_route(z, 8, softmax, bias)
    sure = ref[2] > 1e-6
    assert np.array_equal(ids[sure], ref[0][sure]) and not np.isin(ids, [0, 1, 2, 3, 5]).any()
    if e % 8 == 0:  # runs of which some have no member left
        z[8, : e // 2] = float("-inf")
        ids, w, ref, _ = run_route(z, 6, softmax, ngroups=8, topk_groups=6, group_top=1)
        sure = ref[2] > 1e-6
        assert np.array_equal(ids[sure], ref[0][sure])


def test_route_strides_in_place_outputs_and_no_rows():
    """Logits that are columns of a wider tensor at odd places; outputs given; no rows."""
    import torch
    rng = np.random.default_rng(6)
    wide = torch.from_numpy(rng.standard_normal((77, 300)).astype(np.float32)).cuda()
    for lt in ("f32", "f16", "bf16"):
        z = wide.to(dtype(lt))[:, 5:5 + 129]
        ids, w = torch.full((77, 6), 9, dtype=torch.int32, device="cuda"), torch.full((77, 6), 9.0, device="cuda")
        M.qmm_moe_route(z, 6, ids=ids, weights=w)
        a, b = M.qmm_moe_route(z.contiguous(), 6)
        assert torch.equal(ids, a) and torch.equal(w, b)
    ids, w = M.qmm_moe_route(torch.empty(0, 64, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_route_offsets_past_32_bits():
    import torch
    rng = np.random.default_rng(8)
    ld = (1 << 31) + 32
    store = torch.empty(2 * ld + 128, dtype=torch.float16, device="cuda")
    z = store.as_strided((3, 128), (ld, 1))
    z.copy_(torch.from_numpy(rng.standard_normal((3, 128)).astype(np.float32)))
    a, b = M.qmm_moe_route(z, 8), M.qmm_moe_route(z.contiguous(), 8)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ dispatch

def run_dispatch(ids, e):
    import torch
    n, k = ids.shape
    g = min(e, n * k)
    outs = [torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((n * k,), (n, k), (e + 1,), (g,), (g + 1,))]
    M.qmm_moe_dispatch(dev(ids), e, *outs)
    return [host(t) for t in outs]


def check_dispatch(ids, e):
    for name, got, want in zip(("sorted_tok", "row_idx", "expert_off", "group_expert", "group_off"), run_dispatch(ids, e), R.dispatch(ids, e)):
        assert np.array_equal(got, want), name


@pytest.mark.parametrize("n,k,e", [(1, 1, 1), (1, 8, 128), (8, 8, 128), (7, 3, 5), (64, 1, 2), (65, 8, 1024), (1000, 8, 128), (517, 6, 60),
                                   (8192, 8, 128), (4099, 16, 333), (33, 64, 77), (20000, 4, 1000), (150001, 2, 17), (3, 5, 700),
                                   (100000, 12, 256)])
def test_dispatch(n, k, e):
    """Popular and unpopular experts, ids outside the experts on every side, repeated experts of a
    token, experts without entries."""
    print(f"dispatch {n} x {k} of {e}", flush=True)
    rng = np.random.default_rng(n + e)
    p = rng.random(e) ** 3 + 1e-3
    ids = rng.choice(e, size=(n, k), p=p / p.sum()).astype(np.int32)
    check_dispatch(ids, e)
    ids[rng.random((n, k)) < 0.1] = -1
    ids[rng.random((n, k)) < 0.02] = e
    ids[rng.random((n, k)) < 0.02] = np.iinfo(np.int32).max
    ids[rng.random((n, k)) < 0.02] = np.iinfo(np.int32).min
    check_dispatch(ids, e)


def test_dispatch_extremes():
    """All entries on one expert (the first, the last), no entry at all, no token."""
    for e in (1, 128, 1024):
        for v in (0, e - 1, -1):
            check_dispatch(np.full((3000, 8), v, np.int32), e)
            check_dispatch(np.full((2, 8), v, np.int32), e)
    import torch
    out = M.qmm_moe_dispatch(torch.empty(0, 8, dtype=torch.int32, device="cuda"), 16)
    assert [tuple(t.shape) for t in out] == [(0,), (0, 8), (17,), (0,), (1,)]
    assert (out[2] == 0).all() and (out[4] == 0).all()


def test_route_and_dispatch_in_a_graph_and_on_another_stream():
    """The routing step captured once and replayed on new logits between eager work; a stream given."""
    import torch
    rng = np.random.default_rng(12)
    for n in (8, 3000):
        z = dev(rng.standard_normal((n, 128)).astype(np.float32))

        def step(stream=None):
            ids, w = M.qmm_moe_route(z, 8, stream=stream)
            return [ids, w, *M.qmm_moe_dispatch(ids, 128, stream=stream)]

        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        for i in range(3):
            z.copy_(dev(rng.standard_normal((n, 128)).astype(np.float32)))
            want = step()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        side = torch.cuda.Stream()
        got = step(side.cuda_stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
