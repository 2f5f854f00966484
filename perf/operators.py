"""The operators around the quantized products, as measured: the root-mean-square norm with the
residual's addition (`qmm_rmsnorm`, with `qmm_dequantize_q8_1` for its 8-bit output), the routing of
tokens to experts (`qmm_moe_route`), the expert-sorted dispatch of a routing (`qmm_moe_dispatch`) and
the low-rank adapters beside a shared projection (`qmm_lora`).

`own` false: the plain forms, elementary torch operations in 32 bits.  `own` true: the calls a user
makes of the package.  `exact` is each operator's definition in 64 bits.
"""
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token between two layers: the down products' binary32 sum joins the residual, the
        # next products read q8_1
        {"name": "norm 1 token q8_1", "op": "norm", "ntok": 1, "hidden": 2560, "x": "f32", "res": "f32", "y": "", "q8": True},
        # a small decode batch on a binary16 residual, q8_1 for the experts and binary32 for the router
        {"name": "norm 8 tokens q8_1 + f32", "op": "norm", "ntok": 8, "hidden": 2560, "x": "f32", "res": "f16", "y": "f32", "q8": True},
        # a prompt: 8192 tokens, binary16 activations for the prompt GEMMs
        {"name": "norm 8192 tokens f16", "op": "norm", "ntok": 8192, "hidden": 2560, "x": "f32", "res": "f16", "y": "f16", "q8": False},
        # the final norm of ragged rows of odd width, no residual
        {"name": "norm 517 x 1001 bf16", "op": "norm", "ntok": 517, "hidden": 1001, "x": "bf16", "res": "", "y": "bf16", "q8": False},
        # a decode batch's routing: softmax, top-8 of 128
        {"name": "route 8 tokens top-8/128", "op": "route", "ntok": 8, "nexperts": 128, "topk": 8, "logits": "f32", "score": "softmax",
         "bias": False, "ngroups": 1, "topk_groups": 1, "group_top": 1, "renorm": True, "scale": 1.0, "masked": 0},
        # a prompt's routing over the same experts
        {"name": "route 8192 tokens top-8/128", "op": "route", "ntok": 8192, "nexperts": 128, "topk": 8, "logits": "f32", "score": "softmax",
         "bias": False, "ngroups": 1, "topk_groups": 1, "group_top": 1, "renorm": True, "scale": 1.0, "masked": 0},
        # sigmoid scores with a balance bias, 8 groups of 32 experts of which 4 stay, some experts
        # masked and some rows empty (padding)
        {"name": "route 4099 grouped sigmoid", "op": "route", "ntok": 4099, "nexperts": 256, "topk": 8, "logits": "bf16", "score": "sigmoid",
         "bias": True, "ngroups": 8, "topk_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "masked": 3},
        # a decode batch's dispatch, with the groups the grouped decode takes
        {"name": "dispatch 8 x 8", "op": "dispatch", "ntok": 8, "nexperts": 128, "topk": 8, "drop": 0},
        # a prompt's dispatch, a few tokens of padding dropped
        {"name": "dispatch 8192 x 8", "op": "dispatch", "ntok": 8192, "nexperts": 128, "topk": 8, "drop": 100},
        # eight requests decoding one token each on a projection of the decode workload, each its own adapter
        {"name": "lora 8 requests decode", "op": "lora", "ntok": 8, "nseg": 8, "nadapters": 16, "k": 2560, "nrows": 8192, "rank": 16, "x": "f32"},
        # a mixed chunk of ragged requests, ranks 8 to 64 in one call
        {"name": "lora 517 tokens ragged", "op": "lora", "ntok": 517, "nseg": 11, "nadapters": 8, "k": 2560, "nrows": 12288, "rank": 64, "x": "f16"},
        # a prompt of 8192 tokens of six requests
        {"name": "lora 8192 tokens prompt", "op": "lora", "ntok": 8192, "nseg": 6, "nadapters": 8, "k": 2560, "nrows": 8192, "rank": 16, "x": "f16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def _draw(rng):
    op = rng.choice(["norm", "route", "dispatch", "lora"])
    if op == "norm":
        q8 = rng.random() < 0.5
        y = rng.choice(["", "f32", "f16", "bf16"]) if q8 else rng.choice(["f32", "f16", "bf16"])
        hidden = 32 * _log(rng, 2, 256) if q8 or rng.random() < 0.5 else _log(rng, 33, 8191)
        return {"op": op, "ntok": _log(rng, 1, 8192), "hidden": hidden, "x": rng.choice(["f32", "f16", "bf16"]),
                "res": rng.choice(["", "f32", "f16", "bf16"]), "y": y, "q8": q8}
    if op == "route":
        ngroups = rng.choice([1, 1, 4, 8])
        nexperts = ngroups * _log(rng, 8, 512 // ngroups)
        topk_groups = rng.randint(1, ngroups)
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "ntok": _log(rng, 1, 8192), "nexperts": nexperts,
                "topk": rng.randint(1, min(16, topk_groups * (nexperts // ngroups))), "logits": rng.choice(["f32", "f16", "bf16"]),
                "score": score, "bias": score == "sigmoid", "ngroups": ngroups, "topk_groups": topk_groups,
                "group_top": 1 if score == "softmax" or ngroups == 1 else rng.choice([1, 2]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0, 0, 3])}
    if op == "dispatch":
        ntok, nexperts = _log(rng, 1, 8192), _log(rng, 8, 512)
        return {"op": op, "ntok": ntok, "nexperts": nexperts, "topk": rng.randint(1, 8), "drop": rng.choice([0, ntok // 50])}
    ntok = _log(rng, 1, 8192)
    return {"op": op, "ntok": ntok, "nseg": min(ntok, _log(rng, 1, 48)), "nadapters": rng.randint(1, 16), "k": 32 * _log(rng, 8, 192),
            "nrows": _log(rng, 256, 12288), "rank": 8 * rng.randint(1, 12), "x": "f32" if ntok <= 16 else "f16"}


def draw(rng):
    case = _draw(rng)
    most = max((w["bytes"], w["flops"]) for w in (work(c) for c in listed() if c["op"] == case["op"]))
    while work(case)["bytes"] > most[0] or work(case)["flops"] > 8 * most[1] and case["ntok"] > 1:
        case["ntok"] = max(1, case["ntok"] // 2)
        case.update({n: min(case[n], case["ntok"]) for n in ("nseg", "drop") if n in case})
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    globals()["_prepare_" + case["op"]](case, g, s)
    return s


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_norm(c, g, s):
    n, h = c["ntok"], c["hidden"]
    # a residual stream: a few channels much larger than the others, as models learn them
    channel = torch.exp(0.7 * _randn(g, h))
    s["x"] = (0.5 * _randn(g, n, h)).to(DT[c["x"]])
    s["w"] = 1.0 + 0.2 * _randn(g, h)
    s["res"] = (_randn(g, n, h) * channel).to(DT[c["res"]]) if c["res"] else None
    s["res_out"] = torch.empty_like(s["res"]) if c["res"] else None
    s["y"] = torch.empty(n, h, dtype=DT[c["y"]], device="cuda") if c["y"] else None
    s["yq"] = torch.empty(n, h // 32 * 36, dtype=torch.uint8, device="cuda") if c["q8"] else None
    s["yd"] = torch.empty(n, h, dtype=torch.float16, device="cuda") if c["q8"] else None


def _prepare_route(c, g, s):
    n, e, k = c["ntok"], c["nexperts"], c["topk"]
    # some experts are more popular than others; logits as a router's product gives them
    logits = _randn(g, n, e) + 0.7 * _randn(g, e)
    if c["masked"]:
        logits[:, torch.randperm(e, generator=g, device="cuda")[: c["masked"]]] = float("-inf")
        logits[torch.rand(n, generator=g, device="cuda") < 0.01] = float("-inf")
    s["logits"] = logits.to(DT[c["logits"]])
    s["bias"] = 0.1 * _randn(g, e) if c["bias"] else None
    s["ids"] = torch.empty(n, k, dtype=torch.int32, device="cuda")
    s["weights"] = torch.empty(n, k, device="cuda")


def _prepare_dispatch(c, g, s):
    n, e, k = c["ntok"], c["nexperts"], c["topk"]
    logits = _randn(g, n, e) + 0.7 * _randn(g, e)
    ids = torch.argsort(logits, dim=1, descending=True)[:, :k].to(torch.int32)
    if c["drop"]:
        ids[n - c["drop"]:] = -1  # rows of padding at the chunk's end
    s["ids"] = ids.contiguous()
    ng = min(e, n * k)
    for name, size in (("sorted_tok", n * k), ("expert_off", e + 1), ("group_expert", ng), ("group_off", ng + 1)):
        s[name] = torch.empty(size, dtype=torch.int32, device="cuda")
    s["row_idx"] = torch.empty(n, k, dtype=torch.int32, device="cuda")
    s["ws"] = None


def _prepare_lora(c, g, s):
    n, k, r, nrows, na, nseg = c["ntok"], c["k"], c["rank"], c["nrows"], c["nadapters"], c["nseg"]
    s["x"] = _randn(g, n, k).to(DT[c["x"]])
    s["a"] = (_randn(g, na, r, k) / k ** 0.5).half()
    s["b"] = (_randn(g, na, nrows, r) / r ** 0.5).half()
    # an adapter's rank is at most the table's; its factor is alpha / rank
    s["ranks"] = torch.clamp(8 * torch.randint(1, r // 8 + 1, (na,), generator=g, device="cuda"), max=r).to(torch.int32)
    s["ranks"][0] = r
    s["scales"] = 0.5 + torch.rand(na, generator=g, device="cuda")
    cuts = torch.sort(torch.randperm(n - 1, generator=g, device="cuda")[: nseg - 1] + 1)[0] if n > 1 else torch.empty(0, device="cuda")
    ends = torch.tensor([0], device="cuda"), cuts, torch.tensor([n], device="cuda")
    s["seg_off"] = torch.cat(ends).to(torch.int32)
    adapter = torch.randint(0, na, (nseg,), generator=g, device="cuda").to(torch.int32)
    if nseg > 4:
        adapter[3] = -1  # a request without an adapter
    s["seg_adapter"] = adapter
    s["base"] = _randn(g, n, nrows)
    s["y"] = torch.empty_like(s["base"])
    s["ws"] = None


# ------------------------------------------------------------------ one pass

def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["op"]](s)


def _own_norm(s):
    import moe_expert_amd as M
    c = s["case"]
    M.qmm_rmsnorm(s["x"], s["w"], EPS, res=s["res"], res_out=s["res_out"], y=s["y"], yq=s["yq"])
    yd = M.qmm_dequantize_q8_1(s["yq"], c["hidden"], out=s["yd"]) if c["q8"] else None
    return [s["y"], s["res_out"], yd]


def _plain_norm(s):
    c = s["case"]
    r = s["x"].float()
    if s["res"] is not None:
        r = r + s["res"].float()
    y = r * (1.0 / torch.sqrt((r * r).mean(dim=1, keepdim=True) + EPS)) * s["w"]
    yd = None
    if c["q8"]:
        blocks = y.view(c["ntok"], -1, 32)
        d = blocks.abs().amax(dim=2, keepdim=True) / 127.0
        v = torch.where(d > 0, blocks / d, torch.zeros_like(blocks))
        q = torch.sign(v) * torch.floor(v.abs() + 0.5)
        yd = (q * d.half().float()).view(c["ntok"], -1).half()
    return [y.to(DT[c["y"]]) if c["y"] else None, r.to(DT[c["res"]]) if c["res"] else None, yd]


def _own_route(s):
    import moe_expert_amd as M
    c = s["case"]
    score = M.QMM_SCORE_SIGMOID if c["score"] == "sigmoid" else M.QMM_SCORE_SOFTMAX
    return list(M.qmm_moe_route(s["logits"], c["topk"], score=score, bias=s["bias"], ngroups=c["ngroups"], topk_groups=c["topk_groups"],
                                group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"], ids=s["ids"], weights=s["weights"]))


def _plain_route(s):
    c = s["case"]
    n, e = s["logits"].shape
    low = float("-inf")
    logits = s["logits"].float()
    fit = logits > low  # a masked expert is never chosen
    if c["score"] == "softmax":
        top = logits.amax(dim=1, keepdim=True)
        ex = torch.where(fit, torch.exp(logits - torch.where(top > low, top, torch.zeros_like(top))), torch.zeros_like(logits))
        total = ex.sum(dim=1, keepdim=True)
        score = ex / torch.where(total > 0, total, torch.ones_like(total))
        choice = logits  # the scores rise with the logits
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
        choice = score if s["bias"] is None else score + s["bias"]
    choice = torch.where(fit, choice, torch.full_like(choice, low))
    if c["ngroups"] > 1:
        members = torch.sort(choice.view(n, c["ngroups"], -1), dim=2, descending=True)[0]
        group = members[:, :, : c["group_top"]].sum(dim=2)
        stay = torch.sort(group, dim=1, descending=True, stable=True)[1][:, : c["topk_groups"]]
        kept = torch.zeros(n, c["ngroups"], dtype=torch.bool, device=logits.device).scatter(1, stay, True)
        choice = torch.where(kept.repeat_interleave(e // c["ngroups"], dim=1), choice, torch.full_like(choice, low))
    best, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    best, ids = best[:, : c["topk"]], ids[:, : c["topk"]]
    found = best > low
    w = torch.where(found, torch.gather(score, 1, ids), torch.zeros_like(best))
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return [torch.where(found, ids, torch.full_like(ids, -1)).to(torch.int32), w * c["scale"]]


def _own_dispatch(s):
    import moe_expert_amd as M
    c = s["case"]
    if s["ws"] is None:
        s["ws"] = torch.empty(M.qmm_moe_dispatch_workspace(c["ntok"], c["topk"], c["nexperts"]), dtype=torch.uint8, device="cuda")
    return list(M.qmm_moe_dispatch(s["ids"], c["nexperts"], sorted_tok=s["sorted_tok"], row_idx=s["row_idx"], expert_off=s["expert_off"],
                                   group_expert=s["group_expert"], group_off=s["group_off"], ws=s["ws"]))


def _plain_dispatch(s):
    c = s["case"]
    n, k, e = c["ntok"], c["topk"], c["nexperts"]
    dev = s["ids"].device
    ids = s["ids"].reshape(-1).long()
    key = torch.where((ids >= 0) & (ids < e), ids, torch.full_like(ids, e))
    by, order = torch.sort(key, stable=True)
    sorted_tok = torch.where(by < e, order // k, torch.full_like(order, -1))
    place = torch.empty_like(order).scatter(0, order, torch.arange(n * k, device=dev))
    row_idx = torch.where(key < e, place, torch.full_like(place, -1)).view(n, k)
    count = torch.zeros(e + 1, dtype=torch.long, device=dev).scatter_add(0, key, torch.ones_like(key))[:e]
    expert_off = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), count.cumsum(0)])
    ng = min(e, n * k)
    live = torch.sort((count == 0).to(torch.int32), stable=True)[1][:ng]  # the experts with entries first, in order
    used = count[live] > 0
    group_expert = torch.where(used, live, torch.full_like(live, -1))
    group_off = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.where(used, count[live], torch.zeros_like(live)).cumsum(0)])
    return [t.to(torch.int32) for t in (sorted_tok, row_idx, expert_off, group_expert, group_off)]


def _own_lora(s):
    import moe_expert_amd as M
    c = s["case"]
    if s["ws"] is None:
        s["ws"] = torch.empty(M.qmm_lora_workspace(c["ntok"], c["rank"]), dtype=torch.uint8, device="cuda")
    return M.qmm_lora(s["x"], s["a"], s["b"], s["ranks"], s["scales"], s["seg_off"], s["seg_adapter"], s["y"], base=s["base"], ws=s["ws"])


def _plain_lora(s):
    c = s["case"]
    na, r, k, n = c["nadapters"], c["rank"], c["k"], c["ntok"]
    token = torch.arange(n, device=s["x"].device)
    seg = (token[:, None] >= s["seg_off"][None, 1:]).sum(dim=1)
    adapter = s["seg_adapter"][seg].long()
    # every adapter's low-rank values of every token, those of other adapters masked
    live = torch.arange(r, device=token.device)[None, :] < s["ranks"][:, None]
    mine = torch.arange(na, device=token.device)[None, :] == adapter[:, None]
    v = torch.matmul(s["x"].float(), s["a"].float().view(na * r, k).t()).view(n, na, r)
    v = torch.where(mine[:, :, None] & live[None], v * s["scales"][None, :, None], torch.zeros_like(v))
    flat = s["b"].float().permute(0, 2, 1).reshape(na * r, c["nrows"])
    return s["base"] + torch.matmul(v.view(n, na * r), flat)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "norm":
        n = c["ntok"] * c["hidden"]
        moved = n * (SIZE[c["x"]] + 2 * SIZE.get(c["res"], 0) + SIZE.get(c["y"], 0)) + 4 * c["hidden"]
        return {"bytes": moved + (n // 32 * 36 + 2 * n if c["q8"] else 0), "flops": 5 * n}
    if c["op"] == "route":
        n = c["ntok"] * c["nexperts"]
        return {"bytes": n * SIZE[c["logits"]] + 8 * c["ntok"] * c["topk"] + (4 * c["nexperts"] if c["bias"] else 0), "flops": 4 * n}
    if c["op"] == "dispatch":
        n, ng = c["ntok"] * c["topk"], min(c["nexperts"], c["ntok"] * c["topk"])
        return {"bytes": 12 * n + 4 * (c["nexperts"] + 1) + 4 * (2 * ng + 1), "flops": n}
    # the ranks are drawn: three quarters of the table's on average are taken here
    n, r, used = c["ntok"], 0.75 * c["rank"], min(c["nadapters"], c["nseg"])
    moved = n * c["k"] * SIZE[c["x"]] + 8 * n * c["nrows"] + used * 2 * r * (c["k"] + c["nrows"])
    return {"bytes": moved, "flops": 2 * n * r * (c["k"] + c["nrows"])}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    return globals()["_exact_" + case["op"]](case, prepare(case, seed))


def _exact_norm(c, s):
    r = s["x"].double()
    if s["res"] is not None:
        r = r + s["res"].double()
    y = s["w"].double() * r / torch.sqrt(torch.sum(r ** 2, dim=1) / c["hidden"] + EPS)[:, None]
    # the 8-bit output stands for y: its rounding is part of both sides' error
    return [y if c["y"] else None, r if c["res"] else None, y if c["q8"] else None]


def _exact_route(c, s):
    e, per = c["nexperts"], c["nexperts"] // c["ngroups"]
    z = s["logits"].double()
    out = torch.zeros(c["ntok"], c["topk"], dtype=torch.float64, device=z.device)
    ok = ~torch.isneginf(z)
    if c["score"] == "softmax":
        score = torch.nan_to_num(torch.softmax(z, dim=1))
        pick = z.clone()
    else:
        score = torch.sigmoid(z)
        pick = score if s["bias"] is None else score + s["bias"].double()
    pick = pick.masked_fill(~ok, float("-inf"))
    if c["ngroups"] > 1:
        group = torch.stack([torch.topk(pick[:, i * per:(i + 1) * per], c["group_top"], dim=1)[0].sum(1) for i in range(c["ngroups"])], dim=1)
        for i in range(c["ngroups"]):
            better = (group > group[:, i:i + 1]).sum(1) + (group[:, :i] == group[:, i:i + 1]).sum(1)
            pick[better >= c["topk_groups"], i * per:(i + 1) * per] = float("-inf")
    row = torch.arange(c["ntok"], device=z.device)
    for j in range(c["topk"]):
        best = pick.amax(dim=1)
        at = (pick == best[:, None]).to(torch.int8).argmax(dim=1)  # the first of them
        out[:, j] = torch.where(torch.isneginf(best), torch.zeros_like(best), score[row, at])
        pick[row, at] = float("-inf")
    if c["renorm"]:
        out = torch.nan_to_num(out / out.sum(dim=1, keepdim=True))
    return [None, out * c["scale"]]


def _exact_dispatch(c, s):
    return None


def _exact_lora(c, s):
    y = s["base"].double()
    off, adapter, ranks = s["seg_off"].tolist(), s["seg_adapter"].tolist(), s["ranks"].tolist()
    for i, a in enumerate(adapter):
        if a >= 0 and off[i + 1] > off[i]:
            x = s["x"][off[i]:off[i + 1]].double()
            v = x @ s["a"][a, : ranks[a]].double().t()
            y[off[i]:off[i + 1]] += s["scales"][a].double() * (v @ s["b"][a, :, : ranks[a]].double().t())
    return y
