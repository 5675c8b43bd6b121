"""Cases and plain forms of the operators on a prompt's way through latent attention: rotary positions, appending to the paged
cache with norm and rotation on the way, rows of whole requests out of that cache, and attention in its expanded form (keys and
values of every head, one rotary key for all of them).

`run` computes an operator in plain torch operations, or, where `own` is true, through the library.  Lengths follow from the
case alone; values follow from the seed.
"""
import math

import numpy as np
import torch

own = False

WIDTH, VALUE, ROTARY, NOPE = 576, 512, 64, 128      # a cached row: 512 latent + 64 rotary; a head: 128 + 64 for keys, 128 values
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LTYPE = {"bf16": 0, "f32": 1, "f16": 2}
LAYOUT = {"interleaved": 0, "half": 1}
SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
EPS = 1e-6
LARGEST = 8192 * 8193 // 2 * 64                     # (row, key, head) triples of the largest listed attention


def listed():
    return [
        # the queries of one decoded token: the rotary part of 576-wide rows of 64 heads
        dict(name="rope-1", op="rope", N=1, H=64, dim=64, width=576, layout="interleaved", scaling="yarn", dtype="bf16", pad=0, far=160000),
        # the queries of a large prefill batch, 192 values a head
        dict(name="rope-8192", op="rope", N=8192, H=64, dim=64, width=192, layout="interleaved", scaling="yarn", dtype="bf16", pad=0, far=40000),
        # other layout, type, part of the head and number of tokens; rows of a wider buffer
        dict(name="rope-half-2049", op="rope", N=2049, H=3, dim=40, width=72, layout="half", scaling="linear", dtype="f32", pad=4, far=8000),
        # the rows of one verify step: 64 requests, three positions each
        dict(name="append-rope-192", op="append", N=192, page=64, dtype="bf16", norm=True, layout="interleaved", scaling="yarn", far=160000),
        # the rows of a large prefill batch
        dict(name="append-rope-32768", op="append", N=32768, page=64, dtype="bf16", norm=True, layout="interleaved", scaling="none", far=40000),
        # a few short requests in small pages
        dict(name="gather-short", op="gather", B=3, lo=40, hi=500, page=16, dtype="bf16"),
        # the requests of a large batch of chunks, all of their keys
        dict(name="gather-24", op="gather", B=24, lo=700, hi=16384, page=64, dtype="f16"),
        # a few short prompts with few heads: latency
        dict(name="prompt-short", op="prompt", B=3, tlo=30, thi=200, plo=0, phi=0, H=16, dtype="bf16"),
        # the last tokens of a prompt behind a long context: few rows, the keys split over the card
        dict(name="prompt-tail", op="prompt", B=1, tlo=7, thi=7, plo=20011, phi=20011, H=16, dtype="f16"),
        # a batch of prompts of uneven lengths
        dict(name="prompt-batch", op="prompt", B=12, tlo=100, thi=1500, plo=0, phi=0, H=32, dtype="bf16"),
        # two chunks behind earlier ones
        dict(name="prompt-chunk", op="prompt", B=2, tlo=1000, thi=1000, plo=4099, phi=7200, H=64, dtype="f16"),
        # one long prompt from its beginning
        dict(name="prompt-8192", op="prompt", B=1, tlo=8192, thi=8192, plo=0, phi=0, H=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "gather", "prompt", "prompt", "prompt"])
    layout, scaling = rng.choice(["interleaved", "half"]), rng.choice(["none", "linear", "ntk", "yarn"])
    far = _log(rng, 100, 1000000)
    if op == "rope":
        dim = rng.choice([64, 64, 64, 2 * rng.randint(1, 64)])
        H = rng.choice([1, 3, 8, 16, 32, 64, 128])
        return dict(op="rope", N=_log(rng, 1, 8192 * 64 // max(H, 64)), H=H, dim=dim, width=dim + rng.choice([0, 8, 32, 128, 512]),
                    layout=layout, scaling=scaling, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), pad=rng.choice([0, 0, 4, 16]), far=far)
    if op == "append":
        return dict(op="append", N=_log(rng, 1, 32768), page=rng.choice([1, 16, 32, 48, 64, 128]), dtype=rng.choice(["bf16", "f16"]),
                    norm=rng.random() < 0.7, layout=layout, scaling=scaling, far=far)
    if op == "gather":
        hi = _log(rng, 20, 16384)
        return dict(op="gather", B=_log(rng, 1, 24), lo=hi // rng.randint(1, 20), hi=hi, page=rng.choice([1, 16, 32, 48, 64, 128]),
                    dtype=rng.choice(["bf16", "f16"]))
    while True:
        form = rng.choice(["prompt", "chunk", "few"])
        H = rng.choice([1, 8, 16, 32, 64, 96, 128])
        if form == "prompt":
            thi, phi = _log(rng, 1, 8192), 0
        elif form == "chunk":
            thi, phi = _log(rng, 16, 2048), _log(rng, 100, 16384)
        else:
            thi, phi = rng.randint(1, 8), _log(rng, 1000, 32768)
        c = dict(op="prompt", B=_log(rng, 1, 16), tlo=max(1, thi // rng.randint(1, 10)), thi=thi, plo=phi // rng.randint(1, 10), phi=phi,
                 H=H, dtype=rng.choice(["bf16", "f16"]))
        new, seq = _prompt_lengths(c)
        if _triples(c) <= LARGEST and sum(seq) * H <= 1 << 20 and max(sum(new), 1) * H <= 1 << 19:
            return c


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], uneven, the same for every seed."""
    return [lo + int(((i * 0.6180339887 + 0.37) % 1.0) * (hi - lo + 1)) for i in range(n)]


def _prompt_lengths(c):
    """New tokens of each request, its keys (the new ones among them)."""
    new = _spread(c["B"], c["tlo"], c["thi"])
    return new, [p + t for p, t in zip(_spread(c["B"], c["plo"], c["phi"]), new)]


def _triples(c):
    new, seq = _prompt_lengths(c)
    return sum(t * (l - t) + t * (t + 1) // 2 for t, l in zip(new, seq)) * c["H"]


def _pages(n, page):
    return -(-n // page)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# long contexts: 4096 positions stretched by 40 (yarn), by 8 (linear, ntk)
ROPE = {"none": dict(factor=1.0, original=4096.0), "linear": dict(factor=8.0, original=4096.0), "ntk": dict(factor=8.0, original=4096.0),
        "yarn": dict(factor=40.0, original=4096.0)}
BASE, FAST, SLOW = 10000.0, 32.0, 1.0


def _rope_desc(coli, dim, layout, scaling):
    r = ROPE[scaling]
    return coli.coli_rope_desc(dim, LAYOUT[layout], SCALING[scaling], 1.0, BASE, r["factor"], r["original"], FAST, SLOW)


def _frequencies(dim, scaling):
    """Radians a position of each pair, in 64 bits."""
    r = ROPE[scaling]
    factor = r["factor"]
    base = BASE * factor ** (dim / (dim - 2)) if scaling == "ntk" and dim > 2 else BASE
    j = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    f = base ** (-2.0 * j / dim)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":      # pairs that turn often keep their frequency, pairs that turn seldom are stretched, a ramp between them
        low = max(0, math.floor(dim * math.log(r["original"] / (FAST * 2 * math.pi)) / (2 * math.log(BASE))))
        high = min(dim - 1, math.ceil(dim * math.log(r["original"] / (SLOW * 2 * math.pi)) / (2 * math.log(BASE))))
        stretch = ((j - low) / (high - low if high > low else 0.001)).clamp(0, 1)
        f = f * (1 - stretch) + f / factor * stretch
    return f


def _table(dim, layout, scaling):
    """The frequencies as the program keeps them on the GPU for the library's calls."""
    import quantized_expert_ffn_bias_gb300 as coli
    d = _rope_desc(coli, dim, layout, scaling)
    return d, torch.tensor(coli.colibri_rope_frequencies(d), dtype=torch.int64).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = dict(case)
    s = {"case": c}
    if c["op"] == "rope":
        dt, N, H, width = DTYPES[c["dtype"]], c["N"], c["H"], c["width"]
        s["x"] = torch.randn((N, H * width + c["pad"]), generator=g, device="cuda").to(dt)[:, : H * width].unflatten(1, (H, width))
        s["out"] = torch.zeros((N, H, c["dim"]), dtype=dt, device="cuda")
        s["position"] = torch.randint(0, c["far"], (N,), generator=g, device="cuda").to(torch.int32)
        s["f"] = _frequencies(c["dim"], c["scaling"])
        if own:
            s["desc"], s["freq"] = _table(c["dim"], c["layout"], c["scaling"])
    elif c["op"] == "append":
        dt = DTYPES[c["dtype"]]
        n_pages = _pages(c["N"] + c["N"] // 4 + 1, c["page"])
        wide = (torch.randn((c["N"], WIDTH + 64), generator=g, device="cuda") * 2).to(dt)      # the projection's rows: latent, rotary, more
        s["latent"], s["rope"] = wide[:, :VALUE], wide[:, VALUE:WIDTH]
        s["gain"] = 1.0 + 0.2 * torch.randn((VALUE,), generator=g, device="cuda") if c["norm"] else None
        s["slot"] = torch.randperm(n_pages * c["page"], generator=g, device="cuda")[: c["N"]].to(torch.int32)
        s["position"] = torch.randint(0, c["far"], (c["N"],), generator=g, device="cuda").to(torch.int32)
        s["cache"] = torch.randn((n_pages, c["page"], WIDTH), generator=g, device="cuda").to(dt)
        s["count"] = _ints([c["N"]])
        s["f"] = _frequencies(ROTARY, c["scaling"])
        if own:
            s["desc"], s["freq"] = _table(ROTARY, c["layout"], c["scaling"])
    elif c["op"] == "gather":
        dt, page = DTYPES[c["dtype"]], c["page"]
        lens = _spread(c["B"], c["lo"], c["hi"])
        held = [_pages(v, page) for v in lens]
        n_pages, max_pages = sum(held) + 7, max(held) + 1
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        col = torch.arange(max_pages, device="cuda")[None]
        first = torch.tensor([0] + list(np.cumsum(held)[:-1]), device="cuda")[:, None]
        s["table"] = torch.where(col < torch.tensor(held, device="cuda")[:, None], order[(first + col).clamp(max=n_pages - 1)], -1).to(torch.int32)
        s["cache"] = torch.randn((n_pages, page, WIDTH), generator=g, device="cuda").to(dt)
        s["seq"], s["k_start"], s["status"] = _ints(lens), _ints([0] * (c["B"] + 1)), _ints([0])
        s["m"], s["n_pages"], s["max_pages"] = sum(lens), n_pages, max_pages
        s["latent"] = torch.zeros((s["m"], VALUE), dtype=dt, device="cuda")
        s["rope"] = torch.zeros((s["m"], ROTARY), dtype=dt, device="cuda")
    else:
        dt, H = DTYPES[c["dtype"]], c["H"]
        new, seq = _prompt_lengths(c)
        n, m = sum(new), sum(seq)
        s["n"], s["m"], s["new"], s["seq"] = n, m, new, seq
        s["q"] = (torch.randn((n, H, NOPE + ROTARY), generator=g, device="cuda") * 1.5).to(dt)
        s["kv"] = torch.empty((m, H, 2 * NOPE), dtype=dt, device="cuda")                      # the up-projection's rows: keys, values
        for i in range(0, m, 4096):
            s["kv"][i: i + 4096] = torch.randn((min(4096, m - i), H, 2 * NOPE), generator=g, device="cuda").to(dt)
        s["rope"] = torch.randn((m, ROTARY), generator=g, device="cuda").to(dt)
        s["q_start"], s["k_start"] = _ints([0] + list(np.cumsum(new))), _ints([0] + list(np.cumsum(seq)))
        s["out"] = torch.zeros((n, H, NOPE), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((n, H), dtype=torch.float32, device="cuda")
        s["scale"] = (NOPE + ROTARY) ** -0.5
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
    if c["op"] == "rope":
        x, out = s["x"][..., c["width"] - c["dim"]:], s["out"]
        coli.colibri_rope(s["desc"], LTYPE[c["dtype"]], c["N"], None, c["H"], s["position"], s["freq"], x, x.stride(0), x.stride(1),
                          out, out.stride(0), out.stride(1), st)
        return {"out": out}
    if c["op"] == "append":
        d = coli.coli_kv_desc(c["page"], 1, s["cache"].shape[0], LTYPE[c["dtype"]], c["page"] * WIDTH)
        coli.colibri_kv_append_rope(d, s["desc"], c["N"], s["count"], s["latent"], s["latent"].stride(0), s["gain"], EPS, s["rope"],
                                    s["rope"].stride(0), s["position"], s["freq"], s["slot"], s["cache"], st)
        return {"cache": s["cache"]}
    if c["op"] == "gather":
        d = coli.coli_kv_desc(c["page"], s["max_pages"], s["n_pages"], LTYPE[c["dtype"]], c["page"] * WIDTH)
        coli.colibri_kv_gather(d, c["B"], s["m"], s["seq"], s["table"], s["cache"], s["k_start"], s["latent"], VALUE, s["rope"], ROTARY,
                               s["status"], st)
        return {"k_start": s["k_start"], "latent": s["latent"], "rope": s["rope"], "status": s["status"]}
    H, kv = c["H"], s["kv"]
    n = coli.colibri_prompt_attention_workspace_size(c["B"], s["n"], s["m"], H)
    ws = _workspace(n)
    coli.colibri_prompt_attention(LTYPE[c["dtype"]], c["B"], s["n"], s["m"], H, s["scale"], s["q"], s["q"].stride(0), s["q"].stride(1),
                                  kv, kv.stride(0), kv.stride(1), s["rope"], s["rope"].stride(0), kv[..., NOPE:], kv.stride(0), kv.stride(1),
                                  s["q_start"], s["k_start"], s["out"], s["lse"], ws, n, st)
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the plain forms


def _rotated(x, position, f, layout):
    """x [N, ..., dim] in 32 bits, turned by position * f (angles in 64 bits)."""
    angle = position.double()[:, None] * f
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (x.shape[-1] // 2,)
    cos, sin = torch.cos(angle).float().view(shape), torch.sin(angle).float().view(shape)
    if layout == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _rope(s):
    c = s["case"]
    return {"out": _rotated(s["x"][..., c["width"] - c["dim"]:].float(), s["position"], s["f"], c["layout"]).to(DTYPES[c["dtype"]])}


def _append(s):
    c = s["case"]
    latent = s["latent"].float()
    if c["norm"]:
        latent = latent / torch.sqrt((latent * latent).mean(1, keepdim=True) + EPS) * s["gain"]
    row = torch.cat([latent, _rotated(s["rope"].float(), s["position"], s["f"], c["layout"])], 1)
    s["cache"].view(-1, WIDTH)[s["slot"].long()] = row.to(s["cache"].dtype)
    return {"cache": s["cache"]}


def _gather(s):
    page = s["case"]["page"]
    seq = s["seq"].long()
    k_start = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(seq, 0)])
    row = torch.arange(s["m"], device="cuda")
    b = torch.searchsorted(k_start[1:].contiguous(), row, right=True)
    key = row - k_start[b]
    at = s["table"].long()[b, torch.div(key, page, rounding_mode="floor")] * page + key % page
    rows = s["cache"].view(-1, WIDTH)[at]
    return {"k_start": k_start.to(torch.int32), "latent": rows[:, :VALUE].contiguous(), "rope": rows[:, VALUE:].contiguous(),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _prompt(s):
    """Request by request, in blocks of heads and rows whose scores fit in a gigabyte."""
    H, n0, m0 = s["case"]["H"], 0, 0
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    for t, length in zip(s["new"], s["seq"]):
        rope = s["rope"][m0: m0 + length].float().t()
        step = min(t, 2048)
        heads = max(1, min(H, (1 << 28) // (step * length)))
        for h in range(0, H, heads):
            kv = s["kv"][m0: m0 + length, h: h + heads].float()
            k, v = kv[..., :NOPE].permute(1, 2, 0), kv[..., NOPE:].transpose(0, 1)
            for i in range(0, t, step):
                n = min(step, t - i)
                seen = length - t + i + n                              # keys that the block's last row sees
                q = s["q"][n0 + i: n0 + i + n, h: h + heads].float().transpose(0, 1)
                score = (q[..., :NOPE] @ k[..., :seen] + q[..., NOPE:] @ rope[:, :seen]) * s["scale"]
                last = torch.arange(n, device="cuda") + (length - t + i)
                score = torch.where(torch.arange(seen, device="cuda")[None] <= last[:, None], score, -math.inf)
                top = score.amax(-1, keepdim=True)
                p = torch.exp(score - top)
                total = p.sum(-1, keepdim=True)
                rows = slice(n0 + i, n0 + i + n)
                out[rows, h: h + heads] = (p @ v[:, :seen] / total).transpose(0, 1).to(out.dtype)
                lse[rows, h: h + heads] = (top + torch.log(total))[..., 0].t()
        n0, m0 = n0 + t, m0 + length
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"rope": _rope, "append": _append, "gather": _gather, "prompt": _prompt}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work and exact values


def work(case):
    c = case
    if c["op"] == "rope":
        size = 4 if c["dtype"] == "f32" else 2
        values = c["N"] * c["H"] * c["dim"]
        return {"bytes": 2 * values * size + 4 * c["N"] + 4 * c["dim"], "flops": 3 * values}
    if c["op"] == "append":
        return {"bytes": c["N"] * (2 * 2 * WIDTH + 8) + (4 * VALUE if c["norm"] else 0) + 4 * ROTARY,
                "flops": c["N"] * (3 * ROTARY + (4 * VALUE if c["norm"] else 0))}
    if c["op"] == "gather":
        lens = _spread(c["B"], c["lo"], c["hi"])
        return {"bytes": sum(lens) * 2 * 2 * WIDTH + 4 * sum(_pages(v, c["page"]) for v in lens) + 8 * c["B"], "flops": 0}
    new, seq = _prompt_lengths(c)
    n, m, H = sum(new), sum(seq), c["H"]
    return {"bytes": 2 * (n * H * (NOPE + ROTARY + NOPE) + m * (H * 2 * NOPE + ROTARY)) + 4 * n * H, "flops": 2 * _triples(c) * (2 * NOPE + ROTARY)}


def _turned(x, position, dim, layout, scaling):
    """x [N, ..., dim] of 64-bit numpy values, as complex numbers times exp(i angle)."""
    r = ROPE[scaling]
    wave = 2 * np.arange(dim // 2, dtype=np.float64) / dim
    f = np.exp(-wave * math.log(BASE))
    if scaling == "linear":
        f = f / r["factor"]
    elif scaling == "ntk" and dim > 2:
        f = np.exp(-wave * (math.log(BASE) + math.log(r["factor"]) * dim / (dim - 2)))
    elif scaling == "yarn":
        def pair_of(turns):    # the pair that turns so often over the original context
            return dim * math.log(r["original"] / (2 * math.pi * turns)) / (2 * math.log(BASE))
        lo, hi = max(math.floor(pair_of(FAST)), 0), min(math.ceil(pair_of(SLOW)), dim - 1)
        part = np.clip((np.arange(dim // 2) - lo) / (hi - lo if hi > lo else 0.001), 0, 1)
        f = f * (1 - part + part / r["factor"])
    turn = np.exp(1j * position.astype(np.float64)[:, None] * f).reshape((x.shape[0],) + (1,) * (x.ndim - 2) + (-1,))
    if layout == "half":
        z = (x[..., : dim // 2] + 1j * x[..., dim // 2:]) * turn
        return np.concatenate([z.real, z.imag], -1)
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * turn
    return np.stack([z.real, z.imag], -1).reshape(x.shape)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        x = s["x"][..., c["width"] - c["dim"]:].double().cpu().numpy()
        return {"out": _turned(x, s["position"].cpu().numpy(), c["dim"], c["layout"], c["scaling"])}
    if c["op"] == "append":
        cache = s["cache"].double().view(-1, WIDTH).cpu().numpy()
        at = s["slot"].cpu().numpy()
        latent = s["latent"].double().cpu().numpy()
        if c["norm"]:
            latent = latent * s["gain"].double().cpu().numpy() * (np.square(latent).sum(1) / VALUE + EPS)[:, None] ** -0.5
        cache[at, :VALUE] = latent
        cache[at, VALUE:] = _turned(s["rope"].double().cpu().numpy(), s["position"].cpu().numpy(), ROTARY, c["layout"], c["scaling"])
        return {"cache": cache.reshape(s["cache"].shape)}
    if c["op"] == "gather":
        lens, page = _spread(c["B"], c["lo"], c["hi"]), c["page"]
        table, cache = s["table"].cpu().numpy(), s["cache"].view(-1, page, WIDTH)
        rows = []
        for b, length in enumerate(lens):
            pages = torch.from_numpy(table[b, : _pages(length, page)].astype(np.int64)).cuda()
            rows.append(cache[pages].reshape(-1, WIDTH)[:length])
        rows = torch.cat(rows).double()
        return {"k_start": np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), "latent": rows[:, :VALUE], "rope": rows[:, VALUE:],
                "status": np.zeros(1, np.int32)}
    # head by head, in blocks of rows
    H, n0, m0 = c["H"], 0, 0
    out = torch.zeros((s["n"], H, NOPE), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["n"], H), dtype=torch.float64, device="cuda")
    for t, length in zip(s["new"], s["seq"]):
        for h in range(H):
            key = torch.cat([s["kv"][m0: m0 + length, h, :NOPE], s["rope"][m0: m0 + length]], 1).double()
            value = s["kv"][m0: m0 + length, h, NOPE:].double()
            for i in range(0, t, 1024):
                rows = slice(n0 + i, n0 + min(t, i + 1024))
                ends = torch.arange(length - t + i, length - t + min(t, i + 1024), device="cuda") + 1
                a = (s["q"][rows, h].double() @ key[: int(length - t + min(t, i + 1024))].T) * s["scale"]
                a = a.masked_fill(torch.arange(a.shape[1], device="cuda")[None] >= ends[:, None], -math.inf)
                z = torch.logsumexp(a, 1)
                lse[rows, h] = z
                out[rows, h] = torch.exp(a - z[:, None]) @ value[: a.shape[1]]
        n0, m0 = n0 + t, m0 + length
    return {"out": out, "lse": lse}
