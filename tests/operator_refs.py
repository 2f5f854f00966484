"""Plain 64-bit implementations of the norm, routing, dispatch and adapter definitions (numpy), and
the error bounds their tests use.  U is the unit roundoff of binary32."""
import numpy as np

U = 2.0 ** -24
#: half a unit in the last place relative to the value, and the absolute one of the subnormals
HALF_ULP = {"f32": (0.0, 0.0), "f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 2.0 ** -134)}


def rmsnorm(x, res, w, eps):
    """(r, y) in 64 bits."""
    r = x.astype(np.float64) + (0.0 if res is None else res.astype(np.float64))
    with np.errstate(all="ignore"):
        return r, r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps) * w.astype(np.float64)


def rmsnorm_bound(y, hidden, ytype):
    """|error| of y: r once rounded (1 U), the sum of squares with each value in a chain of at most
    hidden/64 additions and a tree of at most 16 levels (halved by the root), the mean, the root,
    the quotient and two products (8 U), and the output's own rounding."""
    rel, tiny = HALF_ULP[ytype]
    f32 = (hidden / 128 + 8 + 9) * U * np.abs(y) + 2.0 ** -149
    return f32 + (np.abs(y) + f32) * rel + tiny


def route(logits, topk, softmax, bias=None, ngroups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0):
    """(ids, weights, margin): margin is the smallest non-zero distance, per row, at which a choice of
    a run or an expert was decided (binary32 scores may decide closer ones the other way)."""
    z = logits.astype(np.float64)
    n, e = z.shape
    ok = ~np.isnan(z) & (z != -np.inf)
    zz = np.where(ok, z, -np.inf)
    with np.errstate(all="ignore"):
        if softmax:
            top = zz.max(axis=1, keepdims=True)
            ex = np.where(ok, np.where(zz == top, 1.0, np.exp(zz - top)), 0.0)
            total = ex.sum(axis=1, keepdims=True)
            s = np.where(total > 0, ex / np.where(total > 0, total, 1.0), 0.0)
        else:
            s = 1.0 / (1.0 + np.exp(-zz))
        by_logit = softmax and bias is None and (ngroups == 1 or group_top == 1)
        c = zz if by_logit else s + (0.0 if bias is None else bias.astype(np.float64))
    c = np.where(ok & ~np.isnan(c), c, -np.inf)
    margin = np.full(n, np.inf)
    ids = np.full((n, topk), -1, np.int32)
    w = np.zeros((n, topk))
    per = e // ngroups
    for t in range(n):
        ct = c[t].copy()
        if ngroups > 1:
            best = -np.sort(-ct.reshape(ngroups, per), axis=1)[:, :group_top]
            g = np.array([-np.inf if np.isinf(b).any() and (b == -np.inf).any() else b.sum() for b in best])
            order = np.argsort(-g, kind="stable")
            if topk_groups < ngroups and not by_logit and g[order[topk_groups]] != -np.inf:
                gap = g[order[topk_groups - 1]] - g[order[topk_groups]]
                if gap > 0:
                    margin[t] = min(margin[t], gap)
            for i in order[topk_groups:]:
                ct[i * per:(i + 1) * per] = -np.inf
        order = np.argsort(-ct, kind="stable")
        found = [i for i in order[:topk] if ct[i] != -np.inf]
        if not by_logit:
            vals = ct[order[:topk + 1]]
            vals = vals[vals != -np.inf]
            gaps = vals[:-1] - vals[1:]
            gaps = gaps[gaps > 0]
            if gaps.size:
                margin[t] = min(margin[t], gaps.min())
        ids[t, :len(found)] = found
        w[t, :len(found)] = s[t, found]
    if renorm:
        total = w.sum(axis=1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), w)
    return ids, w * scale, margin


def route_weight_bound(w, spread):
    """|error| of a weight: the exponential's argument is rounded once (spread U at a distance
    `spread` from the row's largest logit) and its value within 2 units; the sums add at most
    1024 terms in chains of 16 and a tree of 6 levels, for the softmax and for the renormalisation;
    two quotients and the scale."""
    return (2 * spread + 64) * U * np.abs(w) + 1e-37


def dispatch(ids, nexperts):
    """(sorted_tok, row_idx, expert_off, group_expert, group_off), entries in (expert, token, k) order."""
    n, k = ids.shape
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < nexperts)
    order = np.nonzero(ok)[0]
    order = order[np.argsort(flat[order], kind="stable")]
    sorted_tok = np.full(n * k, -1, np.int32)
    sorted_tok[:order.size] = order // k
    row_idx = np.full(n * k, -1, np.int32)
    row_idx[order] = np.arange(order.size)
    count = np.bincount(flat[ok], minlength=nexperts)
    off = np.zeros(nexperts + 1, np.int32)
    off[1:] = np.cumsum(count)
    g = min(nexperts, n * k)
    live = np.nonzero(count)[0]
    ge = np.full(g, -1, np.int32)
    ge[:live.size] = live
    go = np.full(g + 1, order.size, np.int32)
    go[:live.size] = off[live]
    return sorted_tok, row_idx.reshape(n, k), off, ge, go


def lora(x, a, b, ranks, scales, seg_off, seg_adapter, base):
    """(y, bound, written): y in 64 bits, the error bound of each value and the rows that a segment
    holds.  The bound: an inner sum of k exact products with each term in at most k/16 + 16
    additions (48 more for the splits and their tree); the inner value enters the outer product
    2^-20 below the token's largest; the outer sum of at most 256 terms, the scale and the base."""
    ntok, k = x.shape
    y = base.astype(np.float64).copy()
    bound = 2 * U * np.abs(y)
    written = np.zeros(ntok, bool)
    for s in range(len(seg_adapter)):
        o0 = min(max(int(seg_off[s]), 0), ntok)
        o1 = min(max(int(seg_off[s + 1]), o0), ntok)
        i = int(seg_adapter[s])
        written[o0:o1] = True
        if not 0 <= i < a.shape[0] or o1 == o0:
            continue
        r = min(max(int(ranks[i]), 0), a.shape[1])
        if r == 0:
            continue
        xs, ai, bi = x[o0:o1].astype(np.float64), a[i, :r].astype(np.float64), b[i, :, :r].astype(np.float64)
        sc = float(scales[i])
        v = xs @ ai.T
        ev = (k / 16 + 64) * U * (np.abs(xs) @ np.abs(ai).T) + 2.0 ** -20 * np.abs(v).max(axis=1, keepdims=True)
        y[o0:o1] += sc * (v @ bi.T)
        mag = abs(sc) * (np.abs(v) @ np.abs(bi).T)
        bound[o0:o1] += abs(sc) * (ev @ np.abs(bi).T) + (r / 16 + 24) * U * mag + 2 * U * np.abs(y[o0:o1])
    return y, bound + 2.0 ** -149, written
