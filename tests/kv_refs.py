"""Plain 64-bit implementations of the paged key-value cache's definitions (numpy), its layout, and the
error bounds of the attention's tests.  U is the unit roundoff of binary32."""
import numpy as np

import moe_expert_amd as M

U = 2.0 ** -24
LEVELS = np.array([-127, -104, -83, -65, -49, -35, -22, -10, 1, 13, 25, 38, 53, 69, 89, 113], np.float64)
FORMATS = {"f16": M.QMM_F16, "q8_0": M.QMM_Q8_0, "iq4_nl": M.QMM_IQ4_NL}
FACTOR = {"q8_0": 32, "iq4_nl": 16}  # bytes of a block's factors
#: half a unit in the last place relative to the value, and the absolute one of the subnormals
HALF_ULP = {"f32": (2.0 ** -24, 2.0 ** -150), "f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 2.0 ** -134)}


def quantize(x, kind):
    """(codes, scales float16) of binary32 rows [..., dim]: codes [..., dim] integers (q8_0) or indices."""
    b = x.astype(np.float32).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        a = np.abs(b)
        if kind == "q8_0":
            d = a.max(axis=-1) / np.float32(127)
            r = np.where(d[..., None] == 0, np.float32(0), b / d[..., None])
            t = np.trunc(r)
            code = t + np.where(np.abs(r - t) >= 0.5, np.sign(r), 0)
        else:
            first = a.argmax(axis=-1)[..., None]
            d = np.take_along_axis(b, first, -1)[..., 0] / np.float32(-127)
            r = np.where(d[..., None] == 0, np.float32(1), b / d[..., None]).astype(np.float64)
            far = np.abs(r[..., None] - LEVELS)
            code = far.argmin(axis=-1)  # the first, so the lower level, of two equally near
            d = np.where(d == 0, np.float32(0), d)  # a block of zeros has the scale +0, whatever their signs
        return code.astype(np.int64).reshape(x.shape), d.astype(np.float16)


def chunk_bytes(codes, scales, kind):
    """The bytes of a page and head: codes [page, dim], scales [page, nb] (numpy, by a loop over values)."""
    page, dim = codes.shape
    nb = dim // 32
    f = np.zeros((page, nb * FACTOR[kind]), np.uint8)
    for c in range(dim):
        b, i, n = c // 32, c % 32 // 16, c % 16
        if kind == "q8_0":
            f[:, (n * nb + b) * 2 + i] = codes[:, c].astype(np.int8).view(np.uint8)
        else:
            f[:, n * nb + b] |= (codes[:, c].astype(np.uint8) << (4 * i)).astype(np.uint8)
    return np.concatenate([f.reshape(-1), np.ascontiguousarray(scales).view(np.uint8).reshape(-1)])


def chunk_values(raw, kind, page, dim):
    """float64 [page, dim] of a page and head's bytes (or float16 values)."""
    if kind == "f16":
        return raw.reshape(page, dim).astype(np.float64)
    nb = dim // 32
    cut = page * nb * FACTOR[kind]
    f = raw.reshape(-1)[:cut].reshape(page, -1)
    d = np.ascontiguousarray(raw.reshape(-1)[cut:]).view(np.float16).reshape(page, nb).astype(np.float64)
    out = np.empty((page, dim))
    with np.errstate(all="ignore"):
        for c in range(dim):
            b, i, n = c // 32, c % 32 // 16, c % 16
            if kind == "q8_0":
                q = f[:, (n * nb + b) * 2 + i].view(np.int8).astype(np.float64)
            else:
                q = LEVELS[f[:, n * nb + b] >> (4 * i) & 15]
            out[:, c] = d[:, b] * q
    return out


def stored(x, kind):
    """float64 values that binary32 rows read back as."""
    with np.errstate(all="ignore"):
        if kind == "f16":
            return x.astype(np.float32).astype(np.float16).astype(np.float64)
        code, d = quantize(x, kind)
        q = (code if kind == "q8_0" else LEVELS[code]).astype(np.float64)
        return (q.reshape(*d.shape, 32) * d[..., None].astype(np.float64)).reshape(x.shape)


def random_cache(rng, kind, npages, heads, page, dim, scale=1.0):
    """(raw array [npages, heads, page, row], values float64 [npages, heads, page, dim])."""
    x = (scale * rng.standard_normal((npages, heads, page, dim))).astype(np.float32)
    if kind == "f16":
        raw = x.astype(np.float16)
        return raw, raw.astype(np.float64)
    code, d = quantize(x, kind)
    row = (FACTOR[kind] + 2) * dim // 32
    raw = np.stack([chunk_bytes(code[p, h], d[p, h], kind) for p in range(npages) for h in range(heads)])
    return raw.reshape(npages, heads, page, row), stored(x, kind)


def tables(rng, lens, page, npages=None, width=None, missing=-1):
    """pages int32 [nseq, width] of distinct random pages, `missing` past each sequence's end."""
    need = [-(-max(n, 0) // page) for n in lens]
    npages = sum(need) + 2 if npages is None else npages
    width = max(max(need, default=0), 1) if width is None else width
    pool = rng.permutation(npages)[:sum(need)].tolist()
    t = np.full((len(lens), width), missing, np.int32)
    for i, n in enumerate(need):
        t[i, :min(n, width)] = [pool.pop() for _ in range(n)][:width]
    return t, npages


def positions(seg_off, lens, ntok, nseq):
    """(sequence, position) of each token, sequence -1 for tokens of none."""
    seq, pos = np.full(ntok, -1), np.zeros(ntok, np.int64)
    for s in range(nseq):
        a, b = (s, s + 1) if seg_off is None else (min(max(int(seg_off[s]), 0), ntok), min(max(int(seg_off[s + 1]), 0), ntok))
        for t in range(a, b):
            seq[t], pos[t] = s, int(lens[s]) - (b - t)
    return seq, pos


def attend(q, kval, vval, pages, lens, seg_off, page, heads, scale, window):
    """(out, lse, out's bound before its own rounding, lse's bound, written) in 64 bits; kval, vval float64
    [npages, kv heads, page, dim].

    A score's error in log2 units, over w = scale log2(e) sum |q k|: q once scaled (3 U with the factor's own
    roundings), kept in two binary16 parts (4 U, and 2^-38 of the row's largest value times sum |k|), two chains of
    products of a block of 32 and one over the dim/32 blocks, each rounding once a term, the scale and the
    power of two (8): (80 + dim/32) U w.  An exponential: its argument's rounding (2 U of |z| and of the largest
    |z|) and 4 U of its own.  The sums: three products a 32-position step into one accumulator and a
    rescaling, (n/8 + 200) U in all."""
    ntok, dim = q.shape[0], q.shape[1] // heads
    kvh, npages = kval.shape[1], kval.shape[0]
    out, lse = np.zeros((ntok, heads, dim)), np.full((ntok, heads), -np.inf)
    bound, lbound = np.zeros((ntok, heads, dim)), np.zeros((ntok, heads))
    q = q.astype(np.float64).reshape(ntok, heads, dim)
    seq, pos = positions(seg_off, lens, ntok, len(lens))
    log2e = np.log2(np.e)
    with np.errstate(all="ignore"):
        for t in range(ntok):
            if seq[t] < 0:
                continue
            lo = max(0, pos[t] - window + 1) if window else 0
            j = np.arange(lo, min(pos[t] + 1, pages.shape[1] * page))
            if j.size == 0:
                continue
            pg = pages[seq[t], j // page]
            ok = (pg >= 0) & (pg < npages)
            j, pg = j[ok], pg[ok]
            if j.size == 0:
                continue
            for h in range(heads):
                k, v = kval[pg, h // (heads // kvh), j % page], vval[pg, h // (heads // kvh), j % page]
                z = scale * (k @ q[t, h])
                top = z.max()
                e = np.exp(z - top)
                total = e.sum()
                out[t, h] = e @ v / total
                lse[t, h] = np.log(total) + top
                w = abs(scale) * log2e * (np.abs(k) @ np.abs(q[t, h]))
                tiny = 2.0 ** -38 * abs(scale) * log2e * np.abs(q[t, h]).max() * np.abs(k).sum(axis=1)
                z2 = np.abs(z) * log2e
                rel = np.log(2) * ((80 + dim / 32) * U * w + tiny + 2 * U * (z2 + z2.max())) + 4 * U
                p = e / total
                sums = (j.size / 8 + 200) * U
                bound[t, h] = 1.01 * ((p * rel) @ np.abs(v) + np.abs(out[t, h]) * (p @ rel) + sums * (p @ np.abs(v)) + sums * np.abs(out[t, h]))
                lbound[t, h] = 1.01 * (p @ rel + sums + 4 * U * (abs(lse[t, h]) + np.abs(z).max()))
    return out.reshape(ntok, -1), lse, bound.reshape(ntok, -1) + 2.0 ** -140, lbound, seq >= 0
