"""The paged key-value cache of a decode step, as measured: keys and values quantized as they are written
(`qmm_kv_write`), read back (`qmm_kv_read`), and the attention of new tokens over the cache
(`qmm_kv_attend`).

`own` false: the plain forms, elementary torch operations in 32 bits.  `own` true: the calls a user
makes of the package.  `exact` is each operator's definition in 64 bits.

A cache is a tensor of pages, [npages][kv heads][a page's positions]: binary16 rows ("f16"), or rows of
32-value blocks ("q8_0": a binary16 scale and 32 bytes, "iq4_nl": a binary16 scale and 32 indices of four
bits into sixteen levels).  The positions of a page and head of a block format lie in two planes, first
every position's factors, then every position's scales.  The value j = 16 i + n of block b (i = 0, 1)
stands at place (n, b, i) of its position's factors: byte (n nb + b) 2 + i, or, of four bits, byte
n nb + b, i = 0 in its low half.
"""
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = {"f16": 64, "q8_0": 34, "iq4_nl": 18}  # bytes of 32 values
LEVELS = (-127, -104, -83, -65, -49, -35, -22, -10, 1, 13, 25, 38, 53, 69, 89, 113)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of each of eight requests, as the decode products give them, 8-bit keys and 4-bit values
        {"name": "write 8 tokens q8_0 iq4_nl", "op": "write", "nseq": 8, "ntok": 8, "longest": 4000, "x": "f32", "k": "q8_0", "v": "iq4_nl",
         "kv_heads": 4, "dim": 128, "page": 64},
        # the prompts of six requests, from binary16 projections
        {"name": "write 8192 tokens q8_0", "op": "write", "nseq": 6, "ntok": 8192, "longest": 0, "x": "f16", "k": "q8_0", "v": "q8_0",
         "kv_heads": 4, "dim": 128, "page": 64},
        # a ragged chunk behind cached prefixes, small pages, a cache that is not quantized
        {"name": "write 517 tokens f16 ragged", "op": "write", "nseq": 11, "ntok": 517, "longest": 900, "x": "bf16", "k": "f16", "v": "f16",
         "kv_heads": 3, "dim": 96, "page": 16},
        # a cached prompt read back for a product in binary16
        {"name": "read 8192 positions q8_0", "op": "read", "nseq": 1, "ntok": 8192, "longest": 0, "x": "f16", "k": "q8_0", "v": "q8_0",
         "kv_heads": 4, "dim": 128, "page": 64},
        # the ends of five requests, of 4-bit values, narrow heads and small pages
        {"name": "read 1001 positions iq4_nl", "op": "read", "nseq": 5, "ntok": 1001, "longest": 700, "x": "f32", "k": "iq4_nl", "v": "iq4_nl",
         "kv_heads": 5, "dim": 64, "page": 16},
        # the first tokens of one request
        {"name": "attend 1 x 17 f16", "op": "attend", "nseq": 1, "new": 1, "empty": 0, "longest": 17, "ragged": False, "x": "f32", "k": "f16", "v": "f16",
         "heads": 20, "kv_heads": 4, "dim": 128, "page": 64, "window": 0, "lse": False},
        # a decode batch in the middle of its answers, an 8-bit cache, five heads of queries a head of keys
        {"name": "attend 8 x 4096 q8_0", "op": "attend", "nseq": 8, "new": 1, "empty": 0, "longest": 4096, "ragged": False, "x": "f32", "k": "q8_0", "v": "q8_0",
         "heads": 20, "kv_heads": 4, "dim": 128, "page": 64, "window": 0, "lse": False},
        # a large batch of requests of all lengths, binary16 throughout
        {"name": "attend 64 ragged to 8192 f16", "op": "attend", "nseq": 64, "new": 1, "empty": 3, "longest": 8192, "ragged": True, "x": "f16", "k": "f16", "v": "f16",
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "lse": False},
        # one very long request, 8-bit keys and 4-bit values
        {"name": "attend 1 x 131071 q8_0 iq4_nl", "op": "attend", "nseq": 1, "new": 1, "empty": 0, "longest": 131071, "ragged": False, "x": "f32", "k": "q8_0", "v": "iq4_nl",
         "heads": 20, "kv_heads": 4, "dim": 128, "page": 128, "window": 0, "lse": False},
        # four guessed tokens a request checked at once, a sliding window, wide heads
        {"name": "attend 16 x 4 tokens window", "op": "attend", "nseq": 16, "new": 4, "empty": 1, "longest": 5000, "ragged": True, "x": "bf16", "k": "f16", "v": "q8_0",
         "heads": 12, "kv_heads": 2, "dim": 192, "page": 32, "window": 1000, "lse": False},
        # one head of keys for sixteen of queries, 4 bits throughout, the sums for a later join
        {"name": "attend 32 multi-query iq4_nl", "op": "attend", "nseq": 32, "new": 1, "empty": 0, "longest": 6000, "ragged": True, "x": "f32", "k": "iq4_nl", "v": "iq4_nl",
         "heads": 16, "kv_heads": 1, "dim": 256, "page": 64, "window": 0, "lse": True},
        # up to eight tokens a request, every head its own keys, narrow heads
        {"name": "attend 12 x 8 tokens 64 wide", "op": "attend", "nseq": 12, "new": 8, "empty": 1, "longest": 2000, "ragged": True, "x": "f16", "k": "q8_0", "v": "q8_0",
         "heads": 8, "kv_heads": 8, "dim": 64, "page": 16, "window": 0, "lse": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


KV = [("f16", "f16"), ("f16", "q8_0"), ("f16", "iq4_nl"), ("q8_0", "q8_0"), ("q8_0", "iq4_nl"), ("iq4_nl", "iq4_nl")]


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    k, v = rng.choice(KV)
    c = {"op": op, "x": rng.choice(["f32", "f16", "bf16"]), "k": k, "v": v, "dim": rng.choice([64, 96, 128, 128, 192, 256]),
         "page": rng.choice([16, 32, 48, 64, 128, 256]), "kv_heads": rng.randint(1, 8)}
    if op != "attend":
        c["ntok"] = _log(rng, 1, 8192)
        c["nseq"] = min(c["ntok"], _log(rng, 1, 64))
        c["longest"] = rng.choice([0, _log(rng, 16, 8192)])
        most = max(work(l)["bytes"] for l in listed() if l["op"] == op)
        while work(c)["bytes"] > most:
            c["ntok"] = max(1, c["ntok"] // 2)
            c["nseq"] = min(c["nseq"], c["ntok"])
        return c
    c.update({"nseq": _log(rng, 1, 64), "new": rng.choice([1, 1, 1, rng.randint(2, 8)]), "longest": _log(rng, 16, 131072), "ragged": rng.random() < 0.7,
              "window": rng.choice([0, 0, _log(rng, 16, 4096)]), "lse": rng.random() < 0.3, "heads": c["kv_heads"] * _log(rng, 1, 16)})
    c["empty"] = rng.choice([0, c["nseq"] // 8])
    # no more than the largest listed case, and the padded batch of the plain form in bounds
    most = max(work(l)["bytes"] for l in listed() if l["op"] == "attend")
    while work(c)["bytes"] > most or c["nseq"] * c["longest"] * c["kv_heads"] * c["dim"] > 5.4e8:
        c["longest"] = max(c["new"], c["longest"] // 2)
    return c


# ------------------------------------------------------------------ inputs

def _lengths(c):
    """(length, new tokens) of each sequence; the same for every seed, up to their order."""
    n = c["nseq"]
    if c["op"] == "attend":
        lens = [max(c["new"], round(c["longest"] * (i / n) ** 2)) if c["ragged"] else c["longest"] for i in range(n, 0, -1)]
        new = [c["new"] - i % 3 if c["ragged"] and c["new"] > 3 else c["new"] for i in range(n)]
        for i in range(c["empty"]):  # padding of the batch: nothing in the cache
            lens[n - 1 - i] = 0
        return lens, new
    cuts = [round(c["ntok"] * (i / n) ** 1.5) for i in range(n + 1)]
    cuts = [max(x, i) for i, x in enumerate(cuts)]
    cuts = [min(x, c["ntok"] - (n - i)) for i, x in enumerate(cuts)]
    new = [b - a for a, b in zip(cuts, cuts[1:])]
    return [m + round(c["longest"] * (i + 1) / n) for i, m in enumerate(new)], new


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    heads, dim, page = c["kv_heads"], c["dim"], c["page"]
    lens, new = _lengths(c)
    order = torch.randperm(len(lens), generator=torch.Generator().manual_seed(seed)).tolist()
    lens, new = [lens[i] for i in order], [new[i] for i in order]
    width = max(1, max(-(-n // page) for n in lens))
    need = [-(-n // page) for n in lens]
    npages = sum(need) + 3
    # pages of a pool in the order in which requests came by them
    pool = torch.randperm(npages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = pool[at:at + n]
        at += n
    s = {"case": c, "pages": table, "lens": _i32(lens), "seg_off": _i32([sum(new[:i]) for i in range(len(new) + 1)]), "handle": None, "ws": None}
    ntok = sum(new)
    for name in ("k", "v"):
        s[name + "cache"] = torch.zeros(npages, heads, page, BLOCK[c[name]] * dim // 32, dtype=torch.uint8, device="cuda")
        if c[name] == "f16":
            s[name + "cache"] = s[name + "cache"].view(torch.float16)
        # a few channels of the keys are much larger than the others, as models learn them
        channel = torch.exp(0.5 * _randn(g, heads, 1, dim)) if name == "k" else 1.0
        if c["op"] != "write":
            for p in range(0, npages, 256):
                n = min(256, npages - p)
                x = _randn(g, n, heads, page, dim) * channel
                _put(s[name + "cache"][p:p + n], c[name], x)
        else:
            s[name] = (_randn(g, ntok, heads, 1, dim) * channel).reshape(ntok, heads * dim).to(DT[c["x"]])
    if c["op"] == "attend":
        s["q"] = _randn(g, ntok, c["heads"] * dim).to(DT[c["x"]])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(ntok, c["heads"], device="cuda") if c["lse"] else None
    else:
        # what is written is read back in 32 bits, as the values it stands for
        dt = DT[c["x"]] if c["op"] == "read" else torch.float32
        s["kout"], s["vout"] = (torch.empty(ntok, heads * dim, dtype=dt, device="cuda") for _ in range(2))
    return s


# ------------------------------------------------------------------ a cache's rows in elementary operations

def _planes(cache, kind):
    """(factors [npages, heads, page, bytes], scales [npages, heads, page, 2 * blocks]) of a block format, as bytes."""
    npages, heads, page, row = cache.shape
    nb = row // BLOCK[kind]
    flat = cache.view(npages, heads, page * row)
    cut = page * nb * (BLOCK[kind] - 2)
    return flat[:, :, :cut].unflatten(2, (page, -1)), flat[:, :, cut:].unflatten(2, (page, -1))


def _quantize(x, kind):
    """(factor bytes [..., bytes], scale bytes [..., 2 * blocks]) of rows of binary32 values."""
    b = x.view(*x.shape[:-1], -1, 32)
    most = torch.full((1,), 127.0, device=x.device)  # a quotient, where a Python number gives a product by its reciprocal
    if kind == "q8_0":
        d = b.abs().amax(dim=-1, keepdim=True) / most
        r = torch.where(d > 0, b / d, torch.zeros_like(b))
        q = torch.sign(r) * torch.floor(r.abs() + 0.5)
        f = q.to(torch.int8).view(torch.uint8).view(*b.shape[:-1], 2, 16)
        f = f.movedim(-1, -3).reshape(*x.shape)  # (n, b, i)
    else:
        a = b.abs()
        first = (a == a.amax(dim=-1, keepdim=True)).to(torch.int8).argmax(dim=-1, keepdim=True)
        d = torch.gather(b, -1, first) / -most
        r = torch.where(d != 0, b / d, torch.ones_like(b))
        middle = [(lo + hi) / 2 for lo, hi in zip(LEVELS, LEVELS[1:])]  # a tie goes to the lower level
        q = torch.bucketize(r, torch.tensor(middle, device=x.device)).to(torch.uint8).view(*b.shape[:-1], 2, 16)
        f = (q[..., 0, :] | q[..., 1, :] << 4).movedim(-1, -2).reshape(*x.shape[:-1], -1)  # (n, b)
    return f, d.squeeze(-1).half().view(torch.uint8)


def _values(f, scales, kind):
    """Rows of binary32 values of their bytes."""
    d = scales.contiguous().view(torch.float16).float()
    nb = d.shape[-1]
    if kind == "q8_0":
        q = f.contiguous().view(torch.int8).float().view(*f.shape[:-1], 16, nb, 2)
    else:
        b = f.contiguous().view(*f.shape[:-1], 16, nb)
        q = torch.tensor(LEVELS, dtype=torch.float32, device=f.device)[torch.stack([b & 15, b >> 4], dim=-1).int()]
    v = q * d[..., None, :, None]
    return v.movedim(-3, -1).reshape(*f.shape[:-1], 32 * nb)  # (n, b, i) to (b, i, n)


def _put(cache, kind, x):
    """Whole pages of binary32 values."""
    if kind == "f16":
        cache.copy_(x)
        return
    for to, part in zip(_planes(cache, kind), _quantize(x, kind)):
        to.copy_(part)


def _places(s):
    """(page, place in the page) of each token's position."""
    c = s["case"]
    token = torch.arange(sum(_lengths(c)[1]), device=s["lens"].device)
    seq = (token[:, None] >= s["seg_off"][None, 1:]).sum(dim=1)
    at = s["lens"].long()[seq] - s["seg_off"].long()[seq + 1] + token
    return s["pages"].long()[seq, at // c["page"]], at % c["page"]


def _plain_store(s):
    c = s["case"]
    pg, at = _places(s)
    for name in ("k", "v"):
        x = s[name].float().view(-1, c["kv_heads"], c["dim"])
        cache = s[name + "cache"]
        if c[name] == "f16":
            cache[pg, :, at] = x.half()
        else:
            for to, part in zip(_planes(cache, c[name]), _quantize(x, c[name])):
                to[pg, :, at] = part


def _plain_load(s):
    c = s["case"]
    pg, at = _places(s)
    outs = []
    for name in ("k", "v"):
        cache = s[name + "cache"]
        if c[name] == "f16":
            x = cache[pg, :, at].float()
        else:
            f, d = _planes(cache, c[name])
            x = _values(f[pg, :, at], d[pg, :, at], c[name])
        outs.append(x.reshape(x.shape[0], -1).to(s[name + "out"].dtype))
    return outs


# ------------------------------------------------------------------ one pass

def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["op"]](s)


def _handle(s):
    import moe_expert_amd as M
    if s["handle"] is None:
        kind = {"f16": M.QMM_F16, "q8_0": M.QMM_Q8_0, "iq4_nl": M.QMM_IQ4_NL}
        s["handle"] = M.KvCache(kind[s["case"]["k"]], kind[s["case"]["v"]], s["kcache"], s["vcache"])
    return s["handle"]


def _own_write(s):
    import moe_expert_amd as M
    M.qmm_kv_write(_handle(s), s["pages"], s["lens"], s["k"], s["v"], seg_off=s["seg_off"])
    return _own_read(s)


def _plain_write(s):
    _plain_store(s)
    return _plain_load(s)


def _own_read(s):
    import moe_expert_amd as M
    return list(M.qmm_kv_read(_handle(s), s["pages"], s["lens"], k=s["kout"], v=s["vout"], seg_off=s["seg_off"]))


def _plain_read(s):
    return _plain_load(s)


def _own_attend(s):
    import moe_expert_amd as M
    c, cache = s["case"], _handle(s)
    if s["ws"] is None:
        need = M.qmm_kv_attend_workspace(cache, s["q"].shape[0], c["heads"], c["nseq"], s["pages"].shape[1])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return list(M.qmm_kv_attend(s["q"], cache, s["pages"], s["lens"], seg_off=None if c["new"] == 1 else s["seg_off"],
                                scale=c["dim"] ** -0.5, window=c["window"], out=s["out"], lse=s["lse"], ws=s["ws"]))


def _plain_attend(s):
    c = s["case"]
    heads, kv, dim, new = c["heads"], c["kv_heads"], c["dim"], c["new"]
    ntok = s["q"].shape[0]
    off, lens = s["seg_off"].long(), s["lens"].long()
    dev = lens.device
    table = s["pages"].long().clamp(min=0)
    rows = []
    for name in ("k", "v"):  # every sequence's cache in a row, padded to the longest
        cache = s[name + "cache"]
        if c[name] == "f16":
            x = cache[table].float()
        else:
            f, d = _planes(cache, c[name])
            x = _values(f[table], d[table], c[name])
        rows.append(x.transpose(1, 2).reshape(c["nseq"], kv, -1, dim))
    k, v = rows
    count = off[1:] - off[:-1]
    i = torch.arange(new, device=dev)
    q = s["q"].float()[(off[:-1, None] + i).clamp(max=ntok - 1)]  # [nseq, new, heads * dim]
    q = q.view(c["nseq"], new, kv, heads // kv, dim).transpose(1, 2).reshape(c["nseq"], kv, -1, dim)
    score = torch.matmul(q, k.transpose(2, 3)) * dim ** -0.5
    at = (lens - count)[:, None] + i  # the new tokens' positions
    j = torch.arange(k.shape[2], device=dev)
    live = (j <= at[:, :, None]) & (at[:, :, None] >= 0)
    if c["window"]:
        live = live & (j > at[:, :, None] - c["window"])
    live = live[:, None, :, None].expand(-1, -1, -1, heads // kv, -1).reshape(c["nseq"], 1, score.shape[2], -1)
    score = torch.where(live, score, torch.full_like(score, float("-inf")))
    top = score.amax(dim=3, keepdim=True)
    top = torch.where(top > float("-inf"), top, torch.zeros_like(top))
    p = torch.exp(score - top)
    total = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))  # a row without keys gives zeros
    token = torch.arange(ntok, device=dev)
    seq = (token[:, None] >= off[None, 1:]).sum(dim=1)
    back = lambda t: t.view(c["nseq"], kv, new, heads // kv, -1).transpose(1, 2)[seq, token - off[seq]].reshape(ntok, -1)  # noqa: E731
    return [back(o).to(s["q"].dtype), back(torch.log(total) + top) if c["lse"] else None]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    lens, new = _lengths(c)
    row = c["kv_heads"] * c["dim"]
    cached = row // 32 * (BLOCK[c["k"]] + BLOCK[c["v"]])  # bytes of a position
    if c["op"] == "read":
        return {"bytes": c["ntok"] * (cached + 2 * row * SIZE[c["x"]]), "flops": 2 * c["ntok"] * row}
    if c["op"] == "write":  # written, and read back
        return {"bytes": c["ntok"] * (2 * cached + 2 * row * SIZE[c["x"]] + 8 * row), "flops": 8 * c["ntok"] * row}
    seen, pairs = 0, 0
    for n, m in zip(lens, new):
        for i in range(m):
            at = n - m + i
            if at >= 0:
                pairs += min(at + 1, c["window"] or at + 1)
        first = max(0, n - m)
        seen += n - (max(0, first + 1 - c["window"]) if c["window"] else 0)
    moved = seen * cached + sum(new) * c["heads"] * (2 * c["dim"] * SIZE[c["x"]] + (4 if c["lse"] else 0))
    return {"bytes": moved, "flops": 4 * pairs * c["heads"] * c["dim"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)


def _decoded(s, name, page, first, count):
    """float64 [count, kv heads, dim] of one page, from position `first` of it on."""
    c = s["case"]
    nb = c["dim"] // 32
    chunk = s[name + "cache"][page]
    if c[name] == "f16":
        return chunk[:, first:first + count].double().permute(1, 0, 2)
    per = 32 if c[name] == "q8_0" else 16
    flat = chunk.reshape(c["kv_heads"], -1)
    scale = flat[:, c["page"] * nb * per:].contiguous().view(torch.float16).double().view(-1, c["page"], nb)
    byte = flat[:, : c["page"] * nb * per].reshape(-1, c["page"], 16, nb, per // 16).to(torch.int64)
    out = torch.empty(c["kv_heads"], c["page"], nb, 32, dtype=torch.float64, device=flat.device)
    if c[name] == "q8_0":
        byte = (byte + 128) % 256 - 128
        for i in range(2):
            out[..., 16 * i:16 * i + 16] = byte[..., i].transpose(2, 3).double()
    else:
        level = torch.tensor(LEVELS, dtype=torch.float64, device=flat.device)
        out[..., :16] = level[byte[..., 0] % 16].transpose(2, 3)
        out[..., 16:] = level[byte[..., 0] // 16].transpose(2, 3)
    out = (out * scale[..., None]).reshape(c["kv_heads"], c["page"], -1)
    return out[:, first:first + count].transpose(0, 1)


def _sequence(s, name, i, n):
    """float64 [n, kv heads, dim]: the first n positions of sequence i."""
    page = s["case"]["page"]
    table = s["pages"][i].tolist()
    parts = [_decoded(s, name, table[p // page], 0, min(page, n - p)) for p in range(0, n, page)]
    return torch.cat(parts)


def _exact_read(c, s):
    lens, off = s["lens"].tolist(), s["seg_off"].tolist()
    outs = []
    for name in ("k", "v"):
        parts = [_sequence(s, name, i, lens[i])[lens[i] - (off[i + 1] - off[i]):] for i in range(c["nseq"])]
        outs.append(torch.cat(parts).reshape(c["ntok"], -1))
    return outs


def _exact_write(c, s):
    """The stored values: the scale of a block, its quotients and so its integers are defined in 32 bits (an
    operation in 64, rounded once to 32, is that); the values are their products in 64."""
    outs = []
    for name in ("k", "v"):
        x = s[name].double()
        if c[name] == "f16":
            outs.append(x.half().double())
            continue
        b = x.view(c["ntok"], -1, 32)
        big, at = torch.abs(b).max(dim=2, keepdim=True)
        if c[name] == "q8_0":
            d = (big / 127).float().double()
            r = torch.nan_to_num((b / d).float().double())
            q = torch.trunc(r + 0.5 * torch.sign(r))
        else:
            low = ((torch.abs(b) == big) * torch.arange(32, 0, -1, device=b.device)).argmax(dim=2, keepdim=True)
            d = (torch.gather(b, 2, low) / -127).float().double()
            r = torch.nan_to_num((b / d).float().double())
            level = torch.tensor(LEVELS, dtype=torch.float64, device=b.device)
            q = level[sum((2 * r > lo + hi).long() for lo, hi in zip(LEVELS, LEVELS[1:]))]
        outs.append((q * d.half().double()).reshape(c["ntok"], -1))
    return outs


def _exact_attend(c, s):
    heads, kv, dim = c["heads"], c["kv_heads"], c["dim"]
    lens, off = s["lens"].tolist(), s["seg_off"].tolist()
    ntok = s["q"].shape[0]
    if sum(lens) * heads * dim > 2e10:
        return None
    out = torch.zeros(ntok, heads, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((ntok, heads), float("-inf"), dtype=torch.float64, device="cuda")
    q = s["q"].double().view(ntok, kv, heads // kv, dim)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        k, v = _sequence(s, "k", i, n).transpose(0, 1), _sequence(s, "v", i, n).transpose(0, 1)
        for t in range(off[i], off[i + 1]):
            at = n - (off[i + 1] - t)
            lo = max(0, at + 1 - c["window"]) if c["window"] else 0
            if at < 0:
                continue
            z = q[t] @ k[:, lo:at + 1].transpose(1, 2) / dim ** 0.5
            top = z.max(dim=2, keepdim=True)[0]
            e = torch.exp(z - top)
            out[t] = ((e @ v[:, lo:at + 1]) / e.sum(dim=2, keepdim=True)).view(heads, dim)
            lse[t] = (torch.log(e.sum(dim=2)) + top[:, :, 0]).view(heads)
    return [out.view(ntok, -1), lse if c["lse"] else None]
