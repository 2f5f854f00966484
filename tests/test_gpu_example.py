"""The block of examples/moe_block.py end to end: each step's result against a 64-bit composition on
the dequantized weights, given the routing that the step chose.

The tolerances are relative 2-norms: a prompt step rounds the activations, the weights and H to
binary16 (each within 2^-11), so three roundings, 4 * 2^-11 allowed; a decode step rounds the
activations and H to q8_1, whose step is the block's largest value over 127 (about 2.5 deviations of
32 normal values): an error of 2.5 / 127 / sqrt(12) = 0.6 % each, twice for the experts, 2 %
allowed."""
import numpy as np
import pytest

import moe_expert_amd as M
from tests import operator_refs as R
from tests.gpu_util import host

pytestmark = pytest.mark.gpu


def dense(wtype, w, rows, k):
    return M.qmm_dequant_f16(wtype, w, rows, k).double()


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def reference(b, x, res, off, ad, ids, weights, h=None):
    """Projection with adapters, and the experts' output of the normed h given ids and weights."""
    import torch
    p = x.double() @ dense(M.QMM_IQ4_NL, b.proj, b.hidden, b.hidden).t()
    for s, i in enumerate(ad.tolist()):
        if i >= 0:
            t = slice(int(off[s]), int(off[s + 1]))
            p[t] += float(b.scales[i]) * (x[t].double() @ b.lora_a[i].double().t()) @ b.lora_b[i].double().t()
    r = res.double() + p
    h = r / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-6) * b.norm.double()
    out = torch.zeros_like(p)
    for e in range(b.nexperts):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            g = h[t] @ dense(M.QMM_IQ4_NL, b.gate[e], b.inter, b.hidden).t()
            u = h[t] @ dense(M.QMM_IQ4_NL, b.up[e], b.inter, b.hidden).t()
            y = (g * torch.sigmoid(g) * u) @ dense(M.QMM_Q8_0, b.down[e], b.hidden, b.inter).t()
            out.index_add_(0, t, y * weights[t, k].double()[:, None])
    return p, r, h, out


@pytest.mark.parametrize("path,ntok,lens,adapters", [("decode", 8, [1] * 8, [0, 1, 2, 3, -1, 0, 1, 2]), ("decode", 1, [1], [2]),
                                                     ("prompt", 300, [100, 7, 193], [1, -1, 0])])
def test_block(path, ntok, lens, adapters):
    import torch
    from examples import moe_block as E
    print(f"block {path} {ntok}", flush=True)
    b = E.Block(seed=3, hidden=512, inter=256, nexperts=32, topk=4)
    g = torch.Generator(device="cuda").manual_seed(ntok)
    x = torch.randn(ntok, b.hidden, generator=g, device="cuda")
    x = x.half() if path == "prompt" else x
    res = torch.randn(ntok, b.hidden, generator=g, device="cuda")
    off, ad = E.segments(lens, adapters)
    kept = res.clone()
    out, mid = getattr(b, path)(x, kept, off, ad)
    p, r, h, want = reference(b, x, res, off, ad, mid["ids"], mid["weights"])
    limit = 4 * 2.0 ** -11 if path == "prompt" else 0.02
    assert rel(mid["proj"], p) <= limit and rel(kept, r) <= limit and rel(out, want) <= limit
    assert rel(mid["logits"], h @ dense(M.QMM_Q8_0, b.router, b.nexperts, b.hidden).t()) <= limit
    ids, w, _ = R.route(host(mid["logits"]), b.topk, True)
    assert np.array_equal(host(mid["ids"]), ids)
    assert np.abs(host(mid["weights"]) - w).max() <= 1e-6


def test_block_decode_in_a_graph():
    """A captured decode step replayed on new inputs, between eager steps, equals the eager step."""
    import torch
    from examples import moe_block as E
    b = E.Block(seed=4, hidden=512, inter=256, nexperts=16, topk=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res = torch.randn(4, b.hidden, generator=g, device="cuda"), torch.randn(4, b.hidden, generator=g, device="cuda")
    off, ad = E.segments([1, 1, 2], [0, -1, 3])
    b.decode(x, res.clone(), off, ad)
    kept = res.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = b.decode(x, kept, off, ad)
    for i in range(3):
        x.normal_(generator=g)
        mine = res.clone()
        want, _ = b.decode(x, mine, off, ad)
        kept.copy_(res)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kept, mine)


@pytest.mark.parametrize("path", ["decode", "prompt"])
def test_tokens_without_experts(path):
    """Tokens whose logits are all masked get ids of -1: the dispatch drops them, the products do not
    touch their rows, the combine gives zeros, and the other tokens' results keep their bits."""
    import torch
    from examples import moe_block as E
    b = E.Block(seed=5, hidden=512, inter=256, nexperts=16, topk=4)
    n = 12 if path == "decode" else 200
    g = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(n, b.hidden, generator=g, device="cuda")
    logits = torch.randn(n, b.nexperts, generator=g, device="cuda")
    gone = torch.zeros(n, dtype=torch.bool, device="cuda")
    gone[::3] = True

    def experts(z):
        ids, w = M.qmm_moe_route(z, b.topk)
        tok, row, off, ge, go = M.qmm_moe_dispatch(ids, b.nexperts)
        if path == "decode":
            y, _ = M.qgemv_grouped_experts(M.QMM_IQ4_NL, b.gate, b.up, M.QMM_Q8_0, b.down, b.hidden, b.inter,
                                           M.qmm_quantize_q8_1(h), ge, go, tok, y=torch.zeros(n * b.topk, b.hidden, device="cuda"))
        else:
            y, _ = M.qgemm_prefill_experts(M.QMM_IQ4_NL, b.gate, b.up, M.QMM_Q8_0, b.down, b.nexperts, b.hidden, b.inter, h.half(),
                                           tok, off, y=torch.zeros(n * b.topk, b.hidden, device="cuda"))
        return M.qmm_moe_combine(y, row, w), ids

    full, _ = experts(logits)
    masked = logits.clone()
    masked[gone] = float("-inf")
    some, ids = experts(masked)
    assert (ids[gone] == -1).all() and (some[gone] == 0).all()
    assert torch.equal(some[~gone], full[~gone])
    none, _ = experts(torch.full_like(logits, float("-inf")))
    assert (none == 0).all()
