"""Cases and plain forms of the serving operators around the MoE layer: expert routing from given logits, the paged
compressed cache (block tables and slot maps, appending rows) and attention of new tokens over that cache.

`run` computes an operator in plain torch operations, or, where `own` is true, through the library.  Lengths follow from the
case alone; values follow from the seed.
"""
import math

import numpy as np
import torch

own = False

WIDTH, VALUE = 576, 512          # values a cached token holds (512 latent + 64 rotary); the first 512 are the attention's values
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LTYPE = {"bf16": 0, "f32": 1, "f16": 2}


def listed():
    return [
        # one decoded token of the GLM-class layer (256 experts, top-8) with group-limited routing
        dict(name="route-1", op="route", T=1, E=256, k=8, score="sigmoid", groups=8, keep=4, gscore="top2", renorm=True, bias=True,
             dtype="f32", pad=0),
        # a large prefill batch of the same layer
        dict(name="route-16384", op="route", T=16384, E=256, k=8, score="sigmoid", groups=8, keep=4, gscore="top2", renorm=True,
             bias=True, dtype="f32", pad=0),
        # softmax scores in bf16, no groups, no bias, weights left as they are; rows of a wider buffer; an odd token count
        dict(name="route-softmax-2049", op="route", T=2049, E=160, k=6, score="softmax", groups=1, keep=1, gscore="max",
             renorm=False, bias=False, dtype="bf16", pad=8),
        # one verify step of 64 running requests, three positions each
        dict(name="step-64x3", op="step", B=64, new=3, ragged=False, past=8192, page=64),
        # a mixed batch: 500 requests, most with a token or two, some with long chunks, some finished
        dict(name="step-mixed-500", op="step", B=500, new=256, ragged=True, past=16000, page=16),
        # the rows of one verify step
        dict(name="append-192", op="append", N=192, page=64, dtype="bf16"),
        # the rows of a large prefill batch
        dict(name="append-32768", op="append", N=32768, page=64, dtype="bf16"),
        # a few short requests with few heads: latency
        dict(name="attn-short", op="attn", B=3, T=1, H=16, lo=40, hi=500, page=16, dtype="bf16", topk=0),
        # one request with a long context, one token: the keys split over the card
        dict(name="attn-long", op="attn", B=1, T=1, H=64, lo=65521, hi=65521, page=64, dtype="bf16", topk=0),
        # a verify step: 24 requests of uneven lengths, three positions each
        dict(name="attn-verify", op="attn", B=24, T=3, H=64, lo=700, hi=16384, page=64, dtype="bf16", topk=0),
        # two prefill chunks behind earlier ones
        dict(name="attn-chunk", op="attn", B=2, T=1000, H=64, lo=4099, hi=8200, page=128, dtype="f16", topk=0),
        # sparse attention: every token reads the 2048 keys selected for it
        dict(name="attn-selected", op="attn", B=16, T=3, H=64, lo=20000, hi=65536, page=64, dtype="bf16", topk=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "step", "append", "attn", "attn", "attn"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, 16 // groups), 384 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(16, E // groups * keep))
        return dict(op="route", T=_log(rng, 1, 16384), E=E, k=k, score=rng.choice(["sigmoid", "softmax"]), groups=groups, keep=keep,
                    gscore=rng.choice(["top2", "max"]), renorm=rng.random() < 0.6, bias=rng.random() < 0.6,
                    dtype=rng.choice(["f32", "bf16", "f16"]), pad=rng.choice([0, 0, 3, 8]))
    if op == "step":
        return dict(op="step", B=_log(rng, 1, 1000), new=_log(rng, 1, 256), ragged=rng.random() < 0.5, past=_log(rng, 1, 16000),
                    page=rng.choice([1, 16, 32, 48, 64, 128, 256]))
    if op == "append":
        return dict(op="append", N=_log(rng, 1, 32768), page=rng.choice([1, 16, 32, 48, 64, 128]), dtype=rng.choice(["bf16", "f16"]))
    page, dtype = rng.choice([16, 32, 48, 64, 128]), rng.choice(["bf16", "f16"])
    form = rng.choice(["decode", "decode", "chunk", "selected"])
    if form == "decode":
        B, T, H, hi = _log(rng, 1, 32), rng.randint(1, 4), rng.choice([8, 16, 32, 64, 96, 128]), _log(rng, 100, 16384)
        topk = 0
    elif form == "chunk":
        B, T, H, hi = rng.randint(1, 2), _log(rng, 16, 800), rng.choice([16, 32, 64]), _log(rng, 1000, 8000)
        topk = 0
    else:
        B, T, H, hi = _log(rng, 1, 16), rng.randint(1, 4), rng.choice([16, 64, 128]), _log(rng, 5000, 40000)
        topk = rng.choice([512, 1000, 2048])
    return dict(op="attn", B=B, T=T, H=H, lo=max(T, hi // rng.randint(1, 8)), hi=hi, page=page, dtype=dtype, topk=topk)


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], uneven, the same for every seed."""
    return [lo + int(((i * 0.6180339887 + 0.37) % 1.0) * (hi - lo + 1)) for i in range(n)]


def _attn_lengths(c):
    """Tokens in the cache (the new ones among them) and new tokens of each request."""
    lens = [max(c["T"], v) for v in _spread(c["B"], c["lo"], c["hi"])]
    return lens, [c["T"]] * c["B"]


def _step_lengths(c):
    """Tokens before the step, new tokens (-1: the request has finished)."""
    past = _spread(c["B"], 0, c["past"])
    if not c["ragged"]:
        return past, [c["new"]] * c["B"]
    new = [v if i % 5 == 0 else 1 + v % 3 for i, v in enumerate(_spread(c["B"], 1, c["new"]))]
    return past, [-1 if i % 17 == 11 else 0 if i % 23 == 7 else v for i, v in enumerate(new)]


def _pages(n, page):
    return -(-n // page)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = dict(case)
    s = {"case": c}
    if c["op"] == "route":
        wide = torch.randn((c["T"], c["E"] + c["pad"]), generator=g, device="cuda") * 1.5
        s["logits"] = wide.to(DTYPES[c["dtype"]])
        s["bias"] = torch.randn((c["E"],), generator=g, device="cuda") * (0.1 if c["score"] == "sigmoid" else 0.01) if c["bias"] else None
        s["idx"] = torch.zeros((c["T"], c["k"]), dtype=torch.int32, device="cuda")
        s["w"] = torch.zeros((c["T"], c["k"]), dtype=torch.float32, device="cuda")
    elif c["op"] == "step":
        past, new = _step_lengths(c)
        page = c["page"]
        held = [_pages(v, page) + (1 if i % 9 == 4 else 0) for i, v in enumerate(past)]      # some hold a page of tokens taken back
        need = sum(max(0, _pages(p + n, page) - h) for p, n, h in zip(past, new, held) if n >= 0)
        n_pages = sum(held) + need + 16
        max_pages = max([h for h in held] + [_pages(p + max(n, 0), page) for p, n in zip(past, new)]) + 1
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        row = torch.arange(max_pages, device="cuda")[None, :]
        first = torch.tensor([0] + list(np.cumsum(held)[:-1]), device="cuda")[:, None]
        at = first + row
        table = torch.where(row < torch.tensor(held, device="cuda")[:, None], order[at.clamp(max=n_pages - 1)], -1)
        free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        free[: n_pages - sum(held)] = order[sum(held):]
        n = sum(max(v, 0) for v in new)
        s.update(page=page, max_pages=max_pages, n_pages=n_pages, N=n, new=_ints(new), seq=_ints(past), held=_ints(held),
                 table=table.to(torch.int32).contiguous(), free=free, count=_ints([n_pages - sum(held)]))
        s["seq_out"], s["held_out"], s["count_out"] = _ints([0] * c["B"]), _ints([0] * c["B"]), _ints([0])
        s["q_start"], s["position"], s["slot"] = _ints([0] * (c["B"] + 1)), _ints([0] * n), _ints([0] * n)
        s["status"] = _ints([0])
    elif c["op"] == "append":
        dt = DTYPES[c["dtype"]]
        n_pages = _pages(c["N"] + c["N"] // 4 + 1, c["page"])
        wide = torch.randn((c["N"], WIDTH + 64), generator=g, device="cuda").to(dt)      # the projection's rows: latent, rotary, more
        s["latent"], s["rope"] = wide[:, :VALUE], wide[:, VALUE:WIDTH]
        s["slot"] = torch.randperm(n_pages * c["page"], generator=g, device="cuda")[: c["N"]].to(torch.int32)
        s["cache"] = torch.randn((n_pages, c["page"], WIDTH), generator=g, device="cuda").to(dt)
        s["count"] = _ints([c["N"]])
    else:
        dt, H, page = DTYPES[c["dtype"]], c["H"], c["page"]
        lens, new = _attn_lengths(c)
        n = sum(new)
        total = sum(_pages(v, page) for v in lens)
        n_pages = total + 7
        max_pages = max(_pages(v, page) for v in lens) + 1
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        held = [_pages(v, page) for v in lens]
        row = torch.arange(max_pages, device="cuda")[None, :]
        first = torch.tensor([0] + list(np.cumsum(held)[:-1]), device="cuda")[:, None]
        s["table"] = torch.where(row < torch.tensor(held, device="cuda")[:, None], order[(first + row).clamp(max=n_pages - 1)], -1).to(torch.int32)
        s["cache"] = torch.randn((n_pages, page, WIDTH), generator=g, device="cuda").to(dt)
        s["q"] = (torch.randn((n, H, WIDTH), generator=g, device="cuda") * 1.5).to(dt)
        s["q_start"], s["seq"] = _ints([0] + list(np.cumsum(new))), _ints(lens)
        s["out"] = torch.zeros((n, H, VALUE), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((n, H), dtype=torch.float32, device="cuda")
        s["scale"] = WIDTH ** -0.5
        s["n"], s["longest"], s["max_pages"], s["n_pages"] = n, max(lens), max_pages, n_pages
        s["topk"] = None
        if c["topk"]:       # distinct keys before each token, ascending, -1 behind them, as the key selection gives them
            b = torch.arange(n, device="cuda") // c["T"]
            seen = s["seq"].long()[b] - c["T"] + torch.arange(n, device="cuda") % c["T"] + 1
            score = torch.rand((n, max(lens)), generator=g, device="cuda")
            score = torch.where(torch.arange(max(lens), device="cuda")[None] < seen[:, None], score, -1.0)
            top = score.topk(min(c["topk"], max(lens)), 1)
            key = torch.where(top.values >= 0, top.indices, 1 << 30).sort(1).values
            key = torch.nn.functional.pad(key, (0, c["topk"] - key.shape[1]), value=1 << 30)
            s["topk"] = torch.where(key < 1 << 30, key, -1).to(torch.int32).contiguous()
    return s


# ---------------------------------------------------------------- the library's calls

_work = {}


def _workspace(n):
    """One workspace a program keeps, as large as its largest call asks for."""
    if _work.get("n", 0) < n:
        _work.update(n=n, t=torch.empty(n, dtype=torch.uint8, device="cuda"))
    return _work["t"]


def _own(s):
    import quantized_expert_ffn_bias_gb300 as coli
    c = s["case"]
    st = torch.cuda.current_stream().cuda_stream
    if c["op"] == "route":
        d = coli.coli_route_desc(c["E"], c["k"], {"sigmoid": coli.COLI_SCORE_SIGMOID, "softmax": coli.COLI_SCORE_SOFTMAX}[c["score"]],
                                 c["groups"], c["keep"], {"top2": coli.COLI_GROUP_TOP2, "max": coli.COLI_GROUP_MAX}[c["gscore"]],
                                 1 if c["renorm"] else 0, 2.5)
        coli.colibri_moe_route(d, c["T"], s["logits"], LTYPE[c["dtype"]], c["E"] + c["pad"], s["bias"], s["idx"], s["w"], st)
        return {"idx": s["idx"], "w": s["w"]}
    if c["op"] == "step":
        d = coli.coli_kv_desc(s["page"], s["max_pages"], s["n_pages"], LTYPE["bf16"], s["page"] * WIDTH)
        coli.colibri_kv_step(d, c["B"], s["N"], s["new"], s["seq"], s["held"], s["table"], s["free"], s["count"], s["seq_out"],
                             s["held_out"], s["count_out"], s["q_start"], s["position"], s["slot"], s["status"], st)
        return {k: s[k] for k in ("seq_out", "held_out", "count_out", "table", "free", "q_start", "position", "slot", "status")}
    if c["op"] == "append":
        d = coli.coli_kv_desc(c["page"], 1, s["cache"].shape[0], LTYPE[c["dtype"]], c["page"] * WIDTH)
        coli.colibri_kv_append(d, c["N"], s["count"], s["latent"], s["latent"].stride(0), s["rope"], s["rope"].stride(0), s["slot"],
                               s["cache"], st)
        return {"cache": s["cache"]}
    d = coli.coli_kv_desc(c["page"], s["max_pages"], s["n_pages"], LTYPE[c["dtype"]], c["page"] * WIDTH)
    n = coli.colibri_kv_attention_workspace_size(c["B"], s["n"], c["H"])
    ws = _workspace(n)
    coli.colibri_kv_attention(d, c["B"], s["n"], c["H"], s["scale"], s["q"], c["H"] * WIDTH, WIDTH, s["cache"], s["table"], s["q_start"],
                              s["seq"], s["topk"], c["topk"], s["out"], s["lse"], ws, n, st)
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the plain forms


def _route(s):
    """Scores in 64 bits (they are compared with one another), a stable descending sort (a tie to the lower index)."""
    c = s["case"]
    E, G = c["E"], c["groups"]
    z = s["logits"][:, :E].double()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-z))
    else:
        e = torch.exp(z - z.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    u = p + s["bias"].double() if s["bias"] is not None else p
    if c["keep"] < G:
        ug = u.view(-1, G, E // G)
        best = ug.sort(2, descending=True).values
        gs = best[..., 0] + best[..., 1] if c["gscore"] == "top2" else best[..., 0]
        keep = gs.sort(dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        open_ = torch.zeros(gs.shape, dtype=torch.bool, device=u.device).scatter_(1, keep, True)
        u = torch.where(open_[..., None], ug, -math.inf).view(-1, E)
    idx = u.sort(dim=1, descending=True, stable=True).indices[:, : c["k"]].sort(1).values
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx.to(torch.int32), "w": (w * 2.5).float()}


def _before(v):
    """Exclusive running sum."""
    return torch.cumsum(v, 0) - v


def _step(s):
    page, B, N = s["page"], s["case"]["B"], s["N"]
    new, seq, held = s["new"].long(), s["seq"].long(), s["held"].long()
    table = s["table"]
    dead = new < 0
    add = new.clamp(min=0)
    after = torch.where(dead, 0, seq + add)
    need = torch.where(dead, 0, (torch.div(after + page - 1, page, rounding_mode="floor") - held).clamp(min=0))
    # pages of finished requests go onto the stack of free pages
    col = torch.arange(s["max_pages"], device="cuda")[None]
    back = torch.where(dead, held, 0)
    start = s["count"].long() + _before(back)
    give = dead[:, None] & (col < held[:, None])
    free = torch.nn.functional.pad(s["free"], (0, 1))
    free[torch.where(give, start[:, None] + col, s["n_pages"])] = table
    count = s["count"].long() + back.sum()
    # new pages come off its top, in request order
    take = (col >= held[:, None]) & (col < (held + need)[:, None])
    at = count - 1 - (_before(need)[:, None] + col - held[:, None])
    table = torch.where(take, free[torch.where(take, at, s["n_pages"])], table)
    free = free[: s["n_pages"]]
    q_start = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(add, 0)])
    token = torch.arange(N, device="cuda")
    r = torch.searchsorted(q_start[1:].contiguous(), token, right=True)
    position = seq[r] + token - q_start[r]
    slot = table.long()[r, torch.div(position, page, rounding_mode="floor")] * page + position % page
    i = torch.int32
    return {"seq_out": after.to(i), "held_out": torch.where(dead, 0, held + need).to(i), "count_out": (count - need.sum()).to(i).view(1),
            "table": table, "free": free, "q_start": q_start.to(i), "position": position.to(i), "slot": slot.to(i),
            "status": torch.zeros(1, dtype=i, device="cuda")}


def _append(s):
    rows = s["cache"].view(-1, WIDTH)
    rows[s["slot"].long()] = torch.cat([s["latent"], s["rope"]], 1)
    return {"cache": s["cache"]}


def _softmax_av(score, seen, v):
    """softmax over the seen keys, times the values; 0 and -inf where a row sees none."""
    score = torch.where(seen, score, -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(torch.isinf(m), 0.0, m)), 0.0)
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, (p @ v) / total, 0.0)
    return o, (m + torch.log(total))[..., 0]


def _attn(s):
    c = s["case"]
    B, T, H, page = c["B"], c["T"], c["H"], c["page"]
    rows = s["cache"].view(-1, WIDTH)
    seq, table = s["seq"].long(), s["table"].long()
    if s["topk"] is None:
        key = torch.arange(s["longest"], device="cuda")
        at = (table.clamp(min=0)[:, torch.div(key, page, rounding_mode="floor")] * page + key % page)
        kv = rows[at].float()                                                           # [B, L, 576]
        q = s["q"].view(B, T * H, WIDTH).float()
        pos = (seq[:, None] - T + torch.arange(T, device="cuda")).repeat_interleave(H, 1)
        seen = key[None, None] <= pos[..., None]
    else:
        b = torch.arange(s["n"], device="cuda") // T
        key = s["topk"].long()
        page_of = torch.div(key.clamp(min=0), page, rounding_mode="floor")
        at = table[b[:, None], page_of] * page + key.clamp(min=0) % page
        kv = rows[at].float()                                                           # [tokens, topk, 576]
        q = s["q"].float()
        seen = (key >= 0)[:, None].expand(-1, H, -1)
    o, lse = _softmax_av((q @ kv.transpose(1, 2)) * s["scale"], seen, kv[..., :VALUE])
    return {"out": o.reshape(s["n"], H, VALUE).to(s["out"].dtype), "lse": lse.reshape(s["n"], H)}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "route":
        return _route(state)
    if op == "step":
        return _step(state)
    if op == "append":
        return _append(state)
    return _attn(state)


# ---------------------------------------------------------------- work and exact values


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["T"] * (c["E"] * size + c["k"] * 8) + (4 * c["E"] if c["bias"] else 0), "flops": 10 * c["T"] * c["E"]}
    if c["op"] == "step":
        past, new = _step_lengths(c)
        pages = sum(_pages(p + max(n, 0), c["page"]) - _pages(p, c["page"]) for p, n in zip(past, new))
        n = sum(max(v, 0) for v in new)
        return {"bytes": 24 * c["B"] + 8 * n + 8 * pages + 16, "flops": 8 * n}
    if c["op"] == "append":
        return {"bytes": c["N"] * (2 * 2 * WIDTH + 4), "flops": 0}
    lens, new = _attn_lengths(c)
    n = sum(new)
    if c["topk"]:
        keys = [min(c["topk"], v - c["T"] + t + 1) for v in lens for t in range(c["T"])]
        cached = sum(keys)
    else:
        keys = [v - c["T"] + t + 1 for v in lens for t in range(c["T"])]
        cached = sum(lens)
    return {"bytes": 2 * cached * WIDTH + 2 * n * c["H"] * (WIDTH + VALUE) + 4 * n * c["H"] + (4 * n * c["topk"]),
            "flops": 2 * sum(keys) * c["H"] * (WIDTH + VALUE)}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        z = s["logits"][:, : c["E"]].double().cpu().numpy()
        b = s["bias"].double().cpu().numpy() if s["bias"] is not None else np.zeros(c["E"])
        if c["score"] == "sigmoid":
            p = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        else:
            z = z - z.max(1)[:, None]
            p = np.exp(z) / np.exp(z).sum(1)[:, None]
        u = p + b
        size = c["E"] // c["groups"]
        if c["keep"] < c["groups"]:
            part = np.sort(u.reshape(c["T"], c["groups"], size), 2)
            gs = part[:, :, -1] + (part[:, :, -2] if c["gscore"] == "top2" else 0)
            shut = np.argsort(-gs, 1, kind="stable")[:, c["keep"]:]
            closed = np.zeros((c["T"], c["groups"]), bool)
            np.put_along_axis(closed, shut, True, 1)
            u = np.where(np.repeat(closed, size, 1), -np.inf, u)
        idx = np.sort(np.argsort(-u, 1, kind="stable")[:, : c["k"]], 1)
        w = np.take_along_axis(p, idx, 1)
        return {"idx": idx.astype(np.int32), "w": 2.5 * (w / w.sum(1)[:, None] if c["renorm"] else w)}
    if c["op"] == "step":
        return None
    if c["op"] == "append":
        cache = s["cache"].double().view(-1, WIDTH).cpu().numpy()
        at = s["slot"].cpu().numpy()
        cache[at, :VALUE] = s["latent"].double().cpu().numpy()
        cache[at, VALUE:] = s["rope"].double().cpu().numpy()
        return {"cache": cache.reshape(s["cache"].shape)}
    # token by token where keys were selected, request by request in blocks of tokens else
    T, H, page = c["T"], c["H"], c["page"]
    lens, _ = _attn_lengths(c)
    table, flat = s["table"].cpu().numpy().astype(np.int64), s["cache"].view(-1, WIDTH)
    out = torch.zeros((s["n"], H, VALUE), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["n"], H), dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        keys = np.arange(length)
        where = torch.from_numpy(table[b][keys // page] * page + keys % page).cuda()
        kv = flat[where].double()
        step = 1 if c["topk"] else max(1, (1 << 28) // (length * H))
        for t0 in range(0, T, step):
            t1 = min(T, t0 + step)
            for_rows = slice(b * T + t0, b * T + t1)
            k2 = kv
            if c["topk"]:
                chosen = s["topk"][b * T + t0].long()
                k2 = kv[chosen[chosen >= 0]]
            a = torch.einsum("thd,kd->thk", s["q"][for_rows].double(), k2) * s["scale"]
            if not c["topk"]:
                last = torch.arange(t0, t1, device="cuda") + (length - T)
                a.masked_fill_(torch.arange(length, device="cuda")[None, None] > last[:, None, None], -math.inf)
            z = torch.logsumexp(a, 2)
            lse[for_rows] = z
            out[for_rows] = torch.einsum("thk,kd->thd", torch.exp(a - z[..., None]), k2[:, :VALUE])
    return {"out": out, "lse": lse}
