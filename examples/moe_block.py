"""One decoder block's second half on quantized weights, as a serving loop would run it.

A projection with low-rank adapters (the attention output's), the residual and its norm, the routing,
the dispatch, the experts and the combine, with every intermediate on the GPU:

    decode   q8_1 activations:   qgemv_dense + qmm_lora -> qmm_rmsnorm (q8_1) -> qgemv_dense (router)
             -> qmm_moe_route -> qmm_moe_dispatch -> qgemv_grouped_experts -> qmm_moe_combine
    prompt   binary16 activations: qgemm_dense + qmm_lora -> qmm_rmsnorm (f16) -> qgemm_dense (router)
             -> qmm_moe_route -> qmm_moe_dispatch -> qgemm_prefill_experts -> qmm_moe_combine

The combine's output joins the residual in the next block's qmm_rmsnorm.  No step returns to the
host, so a decode step can be captured in a HIP graph.

    python examples/moe_block.py            random weights, one decode and one prompt step, timed
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch

import moe_expert_amd as M
import synth

EPS = 1e-6


class Block:
    """Random weights of a block: IQ4_NL projection, gate / up and Q8_0 router, down; binary16
    adapters of the projection."""

    def __init__(self, seed=0, hidden=2560, inter=1024, nexperts=128, topk=8, nadapters=4, rank=16, device="cuda"):
        rng = synth.rng_for(seed)
        put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
        self.hidden, self.inter, self.nexperts, self.topk = hidden, inter, nexperts, topk
        small = dict(dlo=1e-4, dhi=1e-3)  # scales that keep the block's values near 1
        self.proj = put(synth.iq4nl_weights(rng, hidden, hidden, **small))
        self.router = put(synth.q8_0_weights(rng, nexperts, hidden, **small))
        self.gate = put(np.stack([synth.iq4nl_weights(rng, inter, hidden, **small) for _ in range(nexperts)]))
        self.up = put(np.stack([synth.iq4nl_weights(rng, inter, hidden, **small) for _ in range(nexperts)]))
        self.down = put(np.stack([synth.q8_0_weights(rng, hidden, inter, **small) for _ in range(nexperts)]))
        self.norm = put(rng.uniform(0.5, 1.5, hidden).astype(np.float32))
        self.lora_a = put((rng.standard_normal((nadapters, rank, hidden)) / hidden ** 0.5).astype(np.float16))
        self.lora_b = put((rng.standard_normal((nadapters, hidden, rank)) / rank ** 0.5).astype(np.float16))
        self.ranks = torch.full((nadapters,), rank, dtype=torch.int32, device=device)
        self.scales = put(rng.uniform(0.2, 0.6, nadapters).astype(np.float32))

    def decode(self, x, residual, seg_off, seg_adapter):
        """x float32 [ntok, hidden] (the attention's output), residual float32 [ntok, hidden], updated
        in place; the tokens seg_off[s] .. seg_off[s+1]-1 use adapter seg_adapter[s].  Returns the
        experts' contribution and the intermediates."""
        b, n = self, x.shape[0]
        xq = M.qmm_quantize_q8_1(x)
        p = M.qgemv_dense(M.QMM_IQ4_NL, b.proj, b.hidden, b.hidden, xq, n)
        M.qmm_lora(x, b.lora_a, b.lora_b, b.ranks, b.scales, seg_off, seg_adapter, p)
        _, hq, _ = M.qmm_rmsnorm(p, b.norm, EPS, res=residual, res_out=residual, yq=True)
        logits = M.qgemv_dense(M.QMM_Q8_0, b.router, b.nexperts, b.hidden, hq, n)
        ids, w = M.qmm_moe_route(logits, b.topk)
        tok, row, _, group_expert, group_off = M.qmm_moe_dispatch(ids, b.nexperts)
        y, _ = M.qgemv_grouped_experts(M.QMM_IQ4_NL, b.gate, b.up, M.QMM_Q8_0, b.down, b.hidden, b.inter, hq, group_expert,
                                       group_off, tok)
        out = M.qmm_moe_combine(y, row, w)
        return out, dict(proj=p, hq=hq, logits=logits, ids=ids, weights=w)

    def prompt(self, x, residual, seg_off, seg_adapter):
        """The same for a chunk of prompt tokens: x float16 [ntok, hidden]."""
        b = self
        p = M.qgemm_dense(M.QMM_IQ4_NL, b.proj, b.hidden, b.hidden, x)
        M.qmm_lora(x, b.lora_a, b.lora_b, b.ranks, b.scales, seg_off, seg_adapter, p)
        h, _, _ = M.qmm_rmsnorm(p, b.norm, EPS, res=residual, res_out=residual, y=torch.float16)
        logits = M.qgemm_dense(M.QMM_Q8_0, b.router, b.nexperts, b.hidden, h)
        ids, w = M.qmm_moe_route(logits, b.topk)
        tok, row, expert_off, _, _ = M.qmm_moe_dispatch(ids, b.nexperts)
        y, _ = M.qgemm_prefill_experts(M.QMM_IQ4_NL, b.gate, b.up, M.QMM_Q8_0, b.down, b.nexperts, b.hidden, b.inter, h, tok,
                                       expert_off)
        out = M.qmm_moe_combine(y, row, w)
        return out, dict(proj=p, h=h, logits=logits, ids=ids, weights=w)


def segments(lengths, adapters, device="cuda"):
    """seg_off, seg_adapter of requests with these many tokens and adapters (-1: none)."""
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return torch.from_numpy(off).to(device), torch.tensor(adapters, dtype=torch.int32, device=device)


def timed(step, reps=10):
    step()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        step()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / reps * 1e3


def main():
    block = Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(8, block.hidden, generator=g, device="cuda")
    res = torch.randn(8, block.hidden, generator=g, device="cuda")
    off, ad = segments([1] * 8, [0, 1, 2, 3, -1, 0, 1, 2])
    step = lambda: block.decode(x, res.clone(), off, ad)  # noqa: E731
    print(f"decode, 8 requests: {timed(step):.1f} us eager", flush=True)
    _, mid = step()
    h = M.qmm_dequantize_q8_1(mid["hq"], block.hidden)  # what the experts read
    y, _, _ = M.qmm_rmsnorm(mid["proj"], block.norm, EPS, res=res, y=torch.float32)
    print(f"decode, q8_1 activations against the binary32 norm: {float((h - y).norm() / y.norm()):.2%}", flush=True)
    graph = torch.cuda.CUDAGraph()
    kept = res.clone()
    with torch.cuda.graph(graph):
        out, _ = block.decode(x, kept, off, ad)
    print(f"decode, 8 requests: {timed(graph.replay):.1f} us from a graph", flush=True)
    x = torch.randn(2048, block.hidden, generator=g, device="cuda").half()
    res = torch.randn(2048, block.hidden, generator=g, device="cuda")
    off, ad = segments([1000, 48, 1000], [0, -1, 3])
    print(f"prompt, 2048 tokens of 3 requests: {timed(lambda: block.prompt(x, res.clone(), off, ad)):.1f} us", flush=True)


if __name__ == "__main__":
    main()
