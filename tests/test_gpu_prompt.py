"""The operators of a prompt's way through latent attention on the GPU (needs a GB300): rotary positions, appending with norm and
rotation, rows out of the paged cache and attention in the expanded form, against 64-bit forms within their error bounds, and a
run of them together with the cache's bookkeeping."""
from __future__ import annotations

import math

import numpy as np
import pytest

from tests import serving_ref as S

pytestmark = pytest.mark.gpu

W, V, ROT = 576, 512, 64
TYPES = {"bf16": 0, "f32": 1, "f16": 2}


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_expert_ffn_bias_gb300 as coli
    coli.build()
    return t


def dt(torch, name):
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def ints(torch, a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def gen(torch, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def within(torch, got, ref, tol, what):
    got = got.double()
    off = (got - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst {float((off / tol).nan_to_num(9e9).max()):.2f} of it"


# ---------------------------------------------------------------- rotary positions


def rope_desc(dim, layout="interleaved", scaling="none", amplitude=1.0, base=10000.0, factor=8.0, original=4096.0):
    import quantized_expert_ffn_bias_gb300 as coli
    return coli.coli_rope_desc(dim, {"interleaved": 0, "half": 1}[layout], {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}[scaling],
                               amplitude, base, factor, original, 32.0, 1.0)


def rope_table(torch, d):
    import quantized_expert_ffn_bias_gb300 as coli
    return torch.tensor(coli.colibri_rope_frequencies(d), dtype=torch.int64).cuda()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype,N,H,dim,before,pad,scaling,amplitude", [
    ("bf16", 1, 64, 64, 512, 0, "yarn", 1.0),        # a decoded token's queries
    ("bf16", 37, 5, 64, 128, 0, "none", 1.0),
    ("f16", 70, 1, 64, 0, 16, "linear", 0.707),
    ("f32", 9, 3, 40, 32, 4, "ntk", 1.25),
    ("bf16", 33, 2, 48, 8, 3, "yarn", 1.0),          # rows that are not whole 16 bytes
    ("f16", 5, 7, 2, 1, 0, "none", 1.0),             # one pair, odd place
    ("f32", 3, 130, 6, 1, 1, "ntk", 1.0),
    ("bf16", 4, 3, 256, 0, 0, "linear", 1.0),
    ("bf16", 300, 128, 64, 128, 0, "yarn", 1.0),     # more heads than a block's pieces
    ("f32", 2, 1024, 4, 0, 0, "none", 1.0),
])
def test_rope(torch, layout, dtype, N, H, dim, before, pad, scaling, amplitude):
    import quantized_expert_ffn_bias_gb300 as coli
    from tests import prompt_ref as R
    t = dt(torch, dtype)
    d = rope_desc(dim, layout, scaling, amplitude)
    freq, g = rope_table(torch, d), gen(torch, N + dim)
    wide = torch.randn((N, H * (before + dim) + pad), generator=g, device="cuda").to(t)
    x = wide[:, : H * (before + dim)].unflatten(1, (H, before + dim))[..., before:]
    pos = torch.randint(-5, 1 << 20, (N,), generator=g, device="cuda").to(torch.int32)
    pos[0] = 2**31 - 1 if N > 2 else 7
    f = R.frequencies(dim, scaling)
    ref, size = R.rotate(x.double(), pos, f, layout, amplitude)
    # the reference's own angles: 2^-52 of position * f
    tol = R.rotate_bound(ref, size, t) + size * (pos.double().abs().view(-1, 1, 1) * 2.0 ** -51)
    out = torch.full((N, H, dim), 7.0, dtype=t, device="cuda")
    coli.colibri_rope(d, TYPES[dtype], N, None, H, pos, freq, x, x.stride(0), x.stride(1), out, out.stride(0), out.stride(1))
    torch.cuda.synchronize()
    within(torch, out, ref, tol, "out of place")
    # in place, some rows not valid: those and what lies beside the part are left alone
    for valid in {N, N // 2, 0}:
        again = wide.clone()
        y = again[:, : H * (before + dim)].unflatten(1, (H, before + dim))[..., before:]
        coli.colibri_rope(d, TYPES[dtype], N, ints(torch, [valid]), H, pos, freq, y, y.stride(0), y.stride(1), y, y.stride(0), y.stride(1))
        torch.cuda.synchronize()
        assert torch.equal(y[:valid], out[:valid])
        y[:valid] = x[:valid]
        assert torch.equal(again, wide)


def test_rope_small_angles_keep_their_bits(torch):
    """Slow pairs at early positions: the sine is as accurate as the angle is, not as a fraction of a turn."""
    import quantized_expert_ffn_bias_gb300 as coli
    d = rope_desc(64, "half", "none", base=1e9)
    freq, pos = rope_table(torch, d), ints(torch, [1, 2, 3])
    x = torch.zeros((3, 1, 64), device="cuda")
    x[..., :32] = 1.0
    out = torch.empty_like(x)
    coli.colibri_rope(d, 1, 3, None, 1, pos, freq, x, 64, 64, out, 64, 64)
    angle = pos.double()[:, None] * 1e9 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    # (the table's own rounding: half a unit of 2^-64 turns of at least 2.4e-10 / 2 pi turns)
    assert ((out[:, 0, 32:].double() - torch.sin(angle)).abs() <= 2.0 ** -21 * torch.sin(angle).abs()).all()


# ---------------------------------------------------------------- append


def append_case(torch, dtype, N, page, layout, gained, seed, spare=9, width=W + 64):
    g = gen(torch, seed)
    t = dt(torch, dtype)
    n_pages = -(-(N + spare) // page)
    wide = (torch.randn((N, width), generator=g, device="cuda") * 3).to(t)
    return dict(latent=wide[:, :V], rope=wide[:, V:W], gain=1 + 0.3 * torch.randn(V, generator=g, device="cuda") if gained else None,
                slot=torch.randperm(n_pages * page, generator=g, device="cuda")[:N].to(torch.int32),
                pos=torch.randint(0, 200000, (N,), generator=g, device="cuda").to(torch.int32),
                cache=torch.randn((n_pages, page, W), generator=g, device="cuda").to(t), n_pages=n_pages)


def call_append(c, kd, rd, freq, N, count, eps, cache, stream=None):
    import quantized_expert_ffn_bias_gb300 as coli
    coli.colibri_kv_append_rope(kd, rd, N, count, c["latent"], c["latent"].stride(0), c["gain"], eps, c["rope"], c["rope"].stride(0),
                                c["pos"], freq, c["slot"], cache, stream)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype,N,page,gained,eps", [("bf16", 1, 64, True, 1e-6), ("f16", 33, 16, True, 1e-5), ("bf16", 515, 1, False, 0.0),
                                                    ("f16", 200, 48, False, 1e-6), ("bf16", 31, 128, True, 0.0)])
def test_append_rope(torch, layout, dtype, N, page, gained, eps):
    import quantized_expert_ffn_bias_gb300 as coli
    from tests import prompt_ref as R
    t = dt(torch, dtype)
    c = append_case(torch, dtype, N, page, layout, gained, N)
    rd = rope_desc(64, layout, "yarn", 1.125)
    freq = rope_table(torch, rd)
    kd = coli.coli_kv_desc(page, 1, c["n_pages"], TYPES[dtype], page * W)
    if N > 20:
        c["slot"][3], c["slot"][17] = -1, c["n_pages"] * page            # rows that go nowhere
    for valid in (N, N // 2):
        cache = c["cache"].clone()
        call_append(c, kd, rd, freq, N, ints(torch, [valid]), eps, cache)
        torch.cuda.synchronize()
        lat = c["latent"].double()
        ref_l = R.norm(lat, c["gain"].double(), eps) if gained else lat
        ref_r, size = R.rotate(c["rope"].double(), c["pos"], R.frequencies(64, "yarn"), layout, 1.125)
        keep = (torch.arange(N, device="cuda") < valid) & (c["slot"] >= 0) & (c["slot"] < c["n_pages"] * page)
        at = c["slot"][keep].long()
        rows = cache.view(-1, W)
        if gained:
            within(torch, rows[at, :V], ref_l[keep], R.norm_bound(ref_l, t)[keep], "latent")
        else:
            assert torch.equal(rows[at, :V], c["latent"][keep])
        tol = R.rotate_bound(ref_r, size, t) + size * c["pos"].double()[:, None] * 2.0 ** -51
        within(torch, rows[at, V:], ref_r[keep], tol[keep], "rotary")
        left = torch.ones(rows.shape[0], dtype=torch.bool, device="cuda")
        left[at] = False
        assert torch.equal(rows[left], c["cache"].view(-1, W)[left])


def test_append_rope_of_layers_that_interleave(torch):
    """Pages of several layers in one buffer: page_stride beyond the page's rows, equal to the same call on a cache of its own."""
    import quantized_expert_ffn_bias_gb300 as coli
    c = append_case(torch, "bf16", 70, 16, "half", True, 5)
    rd = rope_desc(64, "half")
    freq = rope_table(torch, rd)
    alone, both = c["cache"].clone(), torch.zeros((c["n_pages"], 2, 16, W), dtype=torch.bfloat16, device="cuda")
    both[:, 1] = c["cache"]
    call_append(c, coli.coli_kv_desc(16, 1, c["n_pages"], 0, 16 * W), rd, freq, 70, None, 1e-6, alone)
    call_append(c, coli.coli_kv_desc(16, 1, c["n_pages"], 0, 32 * W), rd, freq, 70, None, 1e-6, both.view(-1)[16 * W:])
    torch.cuda.synchronize()
    assert torch.equal(both[:, 1], alone) and not both[:, 0].any()


@pytest.mark.parametrize("dtype,sizes,eps", [("bf16", (1e-38, 3e-30, 1e-16, 1e15, 1e19, 2e36), 0.0), ("bf16", (1e-38, 1e-20, 1e19, 1e36), 1e-6),
                                             ("bf16", (1e-30, 1e-17, 1e-10), 1e-33), ("f16", (6e-8, 1e-4, 6e4), 0.0)])
def test_append_rope_norm_of_any_size(torch, dtype, sizes, eps):
    """Rows whose squares leave fp32's range have their norm all the same; a row of zeros stays one where eps is not 0."""
    import quantized_expert_ffn_bias_gb300 as coli
    from tests import prompt_ref as R
    t, n = dt(torch, dtype), len(sizes)
    c = append_case(torch, dtype, n + 1, 16, "half", True, 3)
    unit = torch.rand((n, V), generator=gen(torch, 4), device="cuda") * 0.9 + 0.1
    wide = torch.zeros((n + 1, V), device="cuda")
    wide[:n] = unit * torch.tensor(sizes, device="cuda")[:, None] if max(sizes) < 1e30 else (unit.double() * torch.tensor(sizes, device="cuda", dtype=torch.float64)[:, None]).float()
    c["latent"] = wide.to(t)
    rd = rope_desc(64, "half")
    cache = c["cache"].clone()
    call_append(c, coli.coli_kv_desc(16, 1, c["n_pages"], TYPES[dtype], 16 * W), rd, rope_table(torch, rd), n + 1, None, eps, cache)
    torch.cuda.synchronize()
    got = cache.view(-1, W)[c["slot"].long(), :V]
    ref = R.norm(c["latent"].double(), c["gain"].double(), eps)
    within(torch, got[:n], ref[:n], R.norm_bound(ref[:n], t), "latent")
    assert torch.isnan(got[n]).all() if eps == 0 else (got[n] == 0).all()


# ---------------------------------------------------------------- gather


def make_table(torch, lens, page, seed, extra=5):
    rng = np.random.default_rng(seed)
    held = [-(-v // page) for v in lens]
    n_pages, max_pages = sum(held) + extra, max(held + [1]) + 1
    order = rng.permutation(n_pages)
    table, at = np.full((len(lens), max_pages), -1, np.int32), 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    return table, n_pages, max_pages


def call_gather(torch, cache, page, stride, table, n_pages, seq, room, wide=0):
    import quantized_expert_ffn_bias_gb300 as coli
    B, max_pages = table.shape
    d = coli.coli_kv_desc(page, max_pages, n_pages, 0, stride)
    lat = torch.full((room + 3, V + wide), 9.0, dtype=torch.bfloat16, device="cuda")
    rot = torch.full((room + 3, ROT + wide), 9.0, dtype=torch.bfloat16, device="cuda")
    start, status = ints(torch, [-7] * (B + 1)), ints(torch, [0])
    coli.colibri_kv_gather(d, B, room, ints(torch, seq), ints(torch, table), cache, start, lat, V + wide, rot, ROT + wide, status)
    torch.cuda.synchronize()
    return lat, rot, start.cpu().numpy(), int(status)


@pytest.mark.parametrize("lens,page,wide,layers", [
    ([1], 64, 0, 1), ([0, 5, 0, 129, 64], 16, 8, 1), ([700, 33, 2000], 48, 0, 2), ([3] * 1000, 1, 0, 1), ([1, 0] * 4096, 16, 0, 1),
    ([30000], 128, 64, 1), ([0, 0], 16, 0, 1)])
def test_gather(torch, lens, page, wide, layers):
    table, n_pages, max_pages = make_table(torch, lens, page, sum(lens))
    cache = torch.randn((n_pages, layers, page, W), generator=gen(torch, 3), device="cuda").to(torch.bfloat16)
    m = sum(lens)
    for room in {m, m + 50, max(0, m - 7)}:
        lat, rot, start, status = call_gather(torch, cache, page, layers * page * W, table, n_pages, lens, room, wide)
        n = min(m, room)
        np.testing.assert_array_equal(start, np.minimum(np.concatenate([[0], np.cumsum(lens)]), room))
        assert status == (S.TOKENS if room < m else 0)
        at = np.concatenate([[table[b, j // page] * page * layers + j % page for j in range(v)] for b, v in enumerate(lens)] + [[]])
        rows = cache.view(-1, W)[torch.tensor(at[:n].astype(np.int64), device="cuda")]
        assert torch.equal(lat[:n, :V], rows[:, :V]) and torch.equal(rot[:n, :ROT], rows[:, V:])
        assert (lat[n:] == 9).all() and (rot[n:] == 9).all() and (lat[:, V:] == 9).all() and (rot[:, ROT:] == 9).all()


def test_gather_reports_bad_pages_and_lengths(torch):
    lens, page = [40, 50, 60, 20], 16
    table, n_pages, max_pages = make_table(torch, lens, page, 1)
    cache = torch.randn((n_pages, page, W), generator=gen(torch, 3), device="cuda").to(torch.bfloat16)
    table[1, 1], table[2, 0] = -1, n_pages
    lat, rot, start, status = call_gather(torch, cache, page, page * W, table, n_pages, lens, 170)
    assert status == S.BAD_PAGE
    zero = (lat[:170, :V] == 0).all(1).cpu().numpy() & (rot[:170] == 0).all(1).cpu().numpy()
    want = np.zeros(170, bool)
    want[40 + 16:40 + 32] = want[90:106] = True
    np.testing.assert_array_equal(zero, want)
    table, n_pages, max_pages = make_table(torch, lens, page, 1)
    lat, rot, start, status = call_gather(torch, cache, page, page * W, table, n_pages, [40, -3, max_pages * page + 5, 20], 200)
    assert status == S.BAD_PAGE | S.TABLE_FULL
    np.testing.assert_array_equal(start, np.cumsum([0, 40, 0, max_pages * page + 5, 20]))
    assert (lat[40 + max_pages * page:45 + max_pages * page, :V] == 0).all()
    huge = call_gather(torch, cache, page, page * W, table, n_pages, [40, 2**31 - 1, 2**31 - 1, 20], 50)
    assert huge[3] & S.TOKENS and list(huge[2]) == [0, 40, 50, 50, 50]


# ---------------------------------------------------------------- attention


def prompt_case(torch, new, seq, H, dtype, seed, spread=1.5, form="joint"):
    """form: how keys and values lie: joint (the up-projection's rows), apart, or heads first."""
    g, t = gen(torch, seed), dt(torch, dtype)
    n, m = sum(new), sum(seq)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    c = dict(new=list(new), seq=list(seq), H=H, dtype=dtype, n=n, m=m, scale=192 ** -0.5)
    c["q"] = (rand(n, H, 192) * spread).to(t)
    if form == "joint":
        kv = rand(max(m, 1), H, 256).to(t)
        c["k"], c["v"] = kv[..., :128], kv[..., 128:]
        c["r"] = rand(max(m, 1), ROT).to(t)
    elif form == "apart":
        c["k"], c["v"] = rand(max(m, 1), H, 136).to(t)[..., 8:], rand(max(m, 1), H, 128).to(t)
        c["r"] = rand(max(m, 1), 80).to(t)[:, 16:]
        c["q"] = torch.cat([c["q"], c["q"]], 2)[..., 192:]
    else:
        c["k"], c["v"] = rand(H, max(m, 1), 128).to(t).transpose(0, 1), rand(H, max(m, 1), 128).to(t).transpose(0, 1)
        c["r"] = rand(max(m, 1), ROT).to(t)
        c["q"] = c["q"].transpose(0, 1).contiguous().transpose(0, 1)
    return c


def call_prompt(torch, c, room=0, stream=None, ws=None, q_start=None, k_start=None, lse=True, out=None):
    import quantized_expert_ffn_bias_gb300 as coli
    H, n = c["H"], c["n"] + room
    q = torch.nn.functional.pad(c["q"], (0, 0, 0, 0, 0, room)) if room else c["q"]
    need = coli.colibri_prompt_attention_workspace_size(len(c["new"]), n, c["m"], H)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        ws.random_(0, 256)                             # what a workspace holds before does not matter
    if out is None:
        out = torch.full((n, H, 128), 7.0, dtype=c["q"].dtype, device="cuda")
    lse_t = torch.full((n, H), 7.0, device="cuda")
    qs = ints(torch, np.concatenate([[0], np.cumsum(c["new"])])) if q_start is None else q_start
    ks = ints(torch, np.concatenate([[0], np.cumsum(c["seq"])])) if k_start is None else k_start
    coli.colibri_prompt_attention(TYPES[c["dtype"]], len(c["new"]), n, c["m"], H, c["scale"], q, q.stride(0), q.stride(1), c["k"],
                                  c["k"].stride(0), c["k"].stride(1), c["r"], c["r"].stride(0), c["v"], c["v"].stride(0), c["v"].stride(1),
                                  qs, ks, out, lse_t if lse else None, ws, ws.numel(), stream)
    return out, lse_t, ws, (q, qs, ks)


def reference(c):
    from tests import prompt_ref as R
    return R.attention(c["q"].double(), c["k"].double(), c["r"].double(), c["v"].double(), c["new"], c["seq"], c["scale"], c["q"].dtype)


def check_prompt(torch, c, **kw):
    import quantized_expert_ffn_bias_gb300 as coli
    out, lse, ws, _ = call_prompt(torch, c, **kw)
    torch.cuda.synchronize()
    assert coli.colibri_kv_check_status(ws) == 0
    ref, ref_lse, tol, tol_lse = reference(c)
    n = c["n"]
    assert torch.isfinite(out[:n]).all()
    within(torch, out[:n], ref, tol, "out")
    none = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse[:n]) & (lse[:n] < 0), none) and (out[:n][none] == 0).all()
    within(torch, lse[:n][~none], ref_lse[~none], tol_lse[~none], "lse")
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,past", [
    ([1], [0]), ([1], [127]), ([1], [128]), ([5], [300]), ([127], [0]), ([128], [0]), ([129], [0]), ([255], [1]), ([256], [0]), ([257], [0]),
    ([300], [0]), ([513], [77]), ([1, 0, 130, 64], [0, 50, 700, 3]), ([640], [1000])])
def test_prompt_lengths(torch, dtype, new, past):
    check_prompt(torch, prompt_case(torch, new, [t + p for t, p in zip(new, past)], 3, dtype, sum(new)))


@pytest.mark.parametrize("new,seq", [([300], [100]), ([10], [0]), ([260, 5], [1, 0]), ([700], [200]), ([3, 400, 2], [0, 0, 9]), ([129], [128])])
def test_prompt_rows_without_keys(torch, new, seq):
    check_prompt(torch, prompt_case(torch, new, seq, 2, "bf16", 11))


def test_prompt_no_keys_at_all(torch):
    c = prompt_case(torch, [5, 300], [0, 0], 2, "bf16", 11)
    out, lse, ws, _ = call_prompt(torch, c)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isinf(lse).all()


@pytest.mark.parametrize("form", ["joint", "apart", "heads"])
@pytest.mark.parametrize("H", [1, 2, 16])
def test_prompt_layouts(torch, form, H):
    check_prompt(torch, prompt_case(torch, [200, 31], [333, 31], H, "bf16", H, form=form), room=9)


@pytest.mark.parametrize("dtype,new,seq,H", [
    ("bf16", [7], [20000], 2),              # few rows: the keys are cut into many parts
    ("f16", [1, 1, 1], [9000, 40, 5000], 5),
    ("bf16", [700], [4000], 32),            # gangs share key tiles
    ("f16", [1024, 300], [1024, 4300], 40),
    ("bf16", [1100], [1100], 64)])
def test_prompt_cut_and_shared_work(torch, dtype, new, seq, H):
    check_prompt(torch, prompt_case(torch, new, seq, H, dtype, H))


def test_prompt_many_requests(torch):
    rng = np.random.default_rng(3)
    new = rng.integers(0, 4, 1500)
    seq = new + rng.integers(0, 60, 1500)
    check_prompt(torch, prompt_case(torch, new.tolist(), seq.tolist(), 2, "bf16", 3))
    new = np.zeros(8192, int)
    new[[0, 5000, 8191]] = [3, 200, 1]
    check_prompt(torch, prompt_case(torch, new.tolist(), (new + 5).tolist(), 1, "bf16", 3))


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prompt_scales(torch, scale, dtype):
    c = prompt_case(torch, [150], [900], 2, dtype, 5)
    c["scale"] = scale
    check_prompt(torch, c)


def test_prompt_references_that_rise(torch):
    """Scores that grow along the keys: every tile raises the reference; and scores far below 0."""
    c = prompt_case(torch, [140], [1500], 2, "f16", 6)
    ramp = torch.linspace(0.0, 6.0, 1500, device="cuda")[:, None]
    c["q"][..., :] = 0.5
    c["k"][:] = (ramp[:, None] + 0.05 * torch.randn((1500, 2, 128), device="cuda")).half()
    check_prompt(torch, c)
    c["k"].neg_()
    check_prompt(torch, c)


def test_prompt_values_that_no_row_sees(torch):
    """Infinities and NaN in keys and values that a row does not see reach neither its output nor its sum."""
    for new, seq in (([200, 64], [450, 64]), ([5], [700]), ([600, 1], [600, 3])):
        c = prompt_case(torch, new, seq, 2, "bf16", 8)
        clean = reference(c)
        # behind every request lies the next one's first key, or the buffer's end: the last row of a request sees only its own
        # keys.  Keys after the middle of each request's new tokens are spoiled: rows before it must not notice.
        first, n0, m0 = [], 0, 0
        for t, s in zip(new, seq):
            spoiled = s - t + t // 2 + (t == 1)
            for i, j in enumerate(range(m0 + min(spoiled, s - 1), m0 + s)):
                what = (math.nan, math.inf, -math.inf)[i % 3]
                c["k"][j, :, i % 128] = what
                c["v"][j, i % 2, (3 * i) % 128] = what
                c["r"][j, i % 64] = what
            first.append(min(spoiled, s - 1) - (s - t))
            n0, m0 = n0 + t, m0 + s
        out, lse, ws, _ = call_prompt(torch, c)
        torch.cuda.synchronize()
        n0 = 0
        for t, f in zip(new, first):
            rows = slice(n0, n0 + max(f, 0))
            within(torch, out[rows], clean[0][rows], clean[2][rows], "rows before the spoiled keys")
            within(torch, lse[rows], clean[1][rows], clean[3][rows], "their sums")
            assert torch.isnan(lse[n0 + max(f, 0):n0 + t]).all(), "rows that see a NaN key"
            n0 += t


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prompt_values_that_some_rows_see(torch, dtype):
    """A value that is not finite reaches exactly the rows that see its key, as itself."""
    c = prompt_case(torch, [300], [500], 2, dtype, 9)
    marks = [(450, 0, 7, math.inf), (451, 1, 100, -math.inf), (460, 0, 33, math.nan), (330, 1, 5, math.inf), (499, 0, 0, math.nan),
             (20, 1, 64, -math.inf)]
    for j, h, x, what in marks:
        c["v"][j, h, x] = what
    out, lse, ws, _ = call_prompt(torch, c)
    torch.cuda.synchronize()
    ref, ref_lse, tol, tol_lse = reference(c)
    want = ref.clone()
    for j, h, x, what in marks:
        want[max(0, j - 200):, h, x] += what
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(out[odd]), torch.isnan(want[odd]))
    assert torch.equal(out[odd].double().nan_to_num(5.0, 6.0, 7.0), want[odd].nan_to_num(5.0, 6.0, 7.0))
    within(torch, out[~odd], ref[~odd], tol[~odd], "the others")
    within(torch, lse, ref_lse, tol_lse, "lse")


def test_prompt_fp16_small_weights_count(torch):
    """Many keys far below the largest: together they weigh as much as it does."""
    c = prompt_case(torch, [2], [9000], 1, "f16", 4)
    c["q"][:] = 0
    c["q"][..., 0] = 1
    c["scale"] = 1.0
    c["k"][:] = 0
    c["k"][..., 0] = -9.0
    c["k"][3, :, 0] = 0.0
    check_prompt(torch, c)


def test_prompt_wrong_starts_compute_nothing(torch):
    import quantized_expert_ffn_bias_gb300 as coli
    c = prompt_case(torch, [40, 50], [60, 70], 2, "bf16", 2)
    for qs, ks in (([0, 60, 50], [0, 60, 130]), ([0, 40, 91], [0, 60, 130]), ([0, 40, 90], [0, 60, 131]), ([-1, 40, 90], [0, 60, 130]),
                   ([0, 40, 90], [0, 131, 130]), ([0, 40, 90], [-2, 60, 130])):
        out, lse, ws, _ = call_prompt(torch, c, q_start=ints(torch, qs), k_start=ints(torch, ks))
        torch.cuda.synchronize()
        assert coli.colibri_kv_check_status(ws) == coli.COLI_DEV_KV_TOKENS
        assert (out == 7).all() and (lse == 7).all()
    # starts that leave rows and keys out at both ends are fine
    out, lse, ws, _ = call_prompt(torch, c, q_start=ints(torch, [3, 40, 80]), k_start=ints(torch, [5, 60, 120]))
    torch.cuda.synchronize()
    assert coli.colibri_kv_check_status(ws) == 0
    assert (out[:3] == 7).all() and (out[80:] == 7).all() and not (out[3:80] == 7).all(-1).any()


def test_prompt_captured_and_on_another_stream(torch):
    """Two captured calls with workspaces of their own, replayed on two streams at once with new inputs, equal eager calls."""
    cs = [prompt_case(torch, [300, 20], [900, 20], 8, "bf16", 1), prompt_case(torch, [7], [5000], 4, "f16", 2)]
    eager = []
    for c in cs:
        out, lse, ws, _ = call_prompt(torch, c)
        eager.append((out, lse))
    torch.cuda.synchronize()
    graphs, outs, held = [], [], []
    for c in cs:
        kept = {k: v.clone() for k, v in c.items() if k in ("q",)}
        qs, ks = ints(torch, np.concatenate([[0], np.cumsum(c["new"])])), ints(torch, np.concatenate([[0], np.cumsum(c["seq"])]))
        import quantized_expert_ffn_bias_gb300 as coli
        ws = torch.empty(coli.colibri_prompt_attention_workspace_size(1, 1, 1, 1), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, lse, _, refs = call_prompt(torch, c, ws=ws, q_start=qs, k_start=ks, stream=torch.cuda.current_stream())
        graphs.append(g)
        outs.append((out, lse))
        held.append((kept, qs, ks, ws, refs))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (a, b), (x, y) in zip(outs, eager):
        assert torch.equal(a, x) and torch.equal(b, y)


def test_prompt_repeats_bit_for_bit(torch):
    c = prompt_case(torch, [500, 70, 9], [3000, 70, 4000], 12, "bf16", 1)
    first = call_prompt(torch, c)
    for _ in range(4):
        again = call_prompt(torch, c, lse=True)
        torch.cuda.synchronize()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    quiet = call_prompt(torch, c, lse=False)
    torch.cuda.synchronize()
    assert torch.equal(first[0], quiet[0]) and (quiet[1] == 7).all()


def test_prompt_wait_that_runs_out(torch):
    """A stage that never counts as there: the waits end, the status says so, the next call is a normal one."""
    import quantized_expert_ffn_bias_gb300 as coli
    c = prompt_case(torch, [300], [2000], 8, "bf16", 1)
    good = call_prompt(torch, c)
    torch.cuda.synchronize()
    coli.colibri_kv_debug_inject(coli.COLI_INJECT_WITHHOLD_STAGE, 20.0)
    try:
        bad = call_prompt(torch, c)
        torch.cuda.synchronize()
        assert coli.colibri_kv_check_status(bad[2]) == coli.COLI_DEV_WAIT_TIMEOUT
    finally:
        coli.colibri_kv_debug_inject(0)
    again = call_prompt(torch, c, ws=bad[2])
    torch.cuda.synchronize()
    assert coli.colibri_kv_check_status(again[2]) == 0
    assert torch.equal(good[0], again[0])


# ---------------------------------------------------------------- together


def test_prompt_steps_together(torch):
    """Prompts, chunks behind them and a finished request through bookkeeping, appending, gathering, the up-projection, the queries'
    rotation and both forms of attention, everything on one stream with lengths that live on the GPU."""
    import quantized_expert_ffn_bias_gb300 as coli
    from tests import prompt_ref as R
    t, page, H, B, eps = torch.float16, 16, 4, 3, 1e-6
    max_pages, n_pages, g = 40, 90, gen(torch, 1)
    kd = coli.coli_kv_desc(page, max_pages, n_pages, coli.COLI_X_F16, page * W)
    rd = rope_desc(ROT, "interleaved", "yarn")
    freq, f = rope_table(torch, rd), R.frequencies(ROT, "yarn")
    cache = torch.zeros((n_pages, page, W), dtype=t, device="cuda")
    table, free = ints(torch, np.full((B, max_pages), -1)), ints(torch, np.arange(n_pages))
    seq, held, count, status = ints(torch, [0] * B), ints(torch, [0] * B), ints(torch, [n_pages]), ints(torch, [0])
    gain = 1 + 0.2 * torch.randn(V, generator=g, device="cuda")
    up_k = (torch.randn((H, 128, V), generator=g, device="cuda") / V ** 0.5).to(t)
    up_v = (torch.randn((H, 128, V), generator=g, device="cuda") / V ** 0.5).to(t)
    scale = 192 ** -0.5
    lens = [0] * B
    for new in ([40, 7, 300], [60, 1, 33], [-1, 5, 0], [9, 0, 260]):
        add = [max(v, 0) for v in new]
        n = sum(add)
        lens = [0 if v < 0 else x + v for x, v in zip(lens, new)]
        m = sum(lens)
        q_start, pos, slot = ints(torch, [0] * (B + 1)), ints(torch, [0] * n), ints(torch, [-1] * n)
        coli.colibri_kv_step(kd, B, n, ints(torch, new), seq, held, table, free, count, seq, held, count, q_start, pos, slot, status)
        raw = (torch.randn((n, W), generator=g, device="cuda") * 2).to(t)
        coli.colibri_kv_append_rope(kd, rd, n, q_start[B:], raw, W, gain, eps, raw[:, V:], W, pos, freq, slot, cache)
        k_start = ints(torch, [0] * (B + 1))
        latent, rope = torch.zeros((m, V), dtype=t, device="cuda"), torch.zeros((m, ROT), dtype=t, device="cuda")
        coli.colibri_kv_gather(kd, B, m, seq, table, cache, k_start, latent, V, rope, ROT, status)
        k = torch.einsum("mv,hdv->mhd", latent.double(), up_k.double()).to(t)
        v = torch.einsum("mv,hdv->mhd", latent.double(), up_v.double()).to(t)
        q_raw = torch.randn((n, H, 192), generator=g, device="cuda").to(t)
        q = q_raw.clone()
        coli.colibri_rope(rd, coli.COLI_X_F16, n, q_start[B:], H, pos, freq, q[..., 128:], H * 192, 192, q[..., 128:], H * 192, 192)
        c = dict(new=add, seq=lens, H=H, dtype="f16", n=n, m=m, scale=scale, q=q, k=k, v=v, r=rope)
        out, lse, ws, _ = call_prompt(torch, c, q_start=q_start, k_start=k_start)
        absorbed = torch.cat([torch.einsum("nhd,hdv->nhv", q[..., :128].double(), up_k.double()).to(t), q[..., 128:]], 2).contiguous()
        out2 = torch.zeros((n, H, V), dtype=t, device="cuda")
        need = coli.colibri_kv_attention_workspace_size(B, n, H)
        ws2 = torch.zeros(need, dtype=torch.uint8, device="cuda")
        coli.colibri_kv_attention(kd, B, n, H, scale, absorbed, H * W, W, cache, table, q_start, seq, None, 0, out2, None, ws2, need)
        torch.cuda.synchronize()
        assert int(status) == 0 and coli.colibri_kv_check_status(ws) == 0 and coli.colibri_kv_check_status(ws2) == 0
        np.testing.assert_array_equal(seq.cpu().numpy(), lens)
        np.testing.assert_array_equal(q_start.cpu().numpy(), np.concatenate([[0], np.cumsum(add)]))
        np.testing.assert_array_equal(k_start.cpu().numpy(), np.concatenate([[0], np.cumsum(lens)]))
        want_pos = np.concatenate([np.arange(x - a, x) for x, a in zip(lens, add)])
        np.testing.assert_array_equal(pos.cpu().numpy(), want_pos)
        # the new rows, as they came out of the cache
        at = torch.tensor(np.concatenate([s0 + np.arange(x - a, x) for s0, x, a in zip(np.cumsum([0] + lens), lens, add)]).astype(np.int64), device="cuda")
        ref = R.norm(raw[:, :V].double(), gain.double(), eps)
        within(torch, latent[at], ref, R.norm_bound(ref, t), "latent")
        ref, size = R.rotate(raw[:, V:].double(), pos, f, "interleaved")
        within(torch, rope[at], ref, R.rotate_bound(ref, size, t) + size * 2.0 ** -40, "rotary keys")
        ref, size = R.rotate(q_raw[..., 128:].double(), pos, f, "interleaved")
        within(torch, q[..., 128:], ref, R.rotate_bound(ref, size, t) + size * 2.0 ** -40, "queries")
        assert torch.equal(q[..., :128], q_raw[..., :128])
        ref, ref_lse, tol, tol_lse = reference(c)
        within(torch, out, ref, tol, "attention")
        within(torch, lse, ref_lse, tol_lse, "lse")
        # the absorbed form: the same weights up to the rounding of k (there of the absorbed query), which moves a score by
        # ds = 2^-11 scale (sum |q||k| + sum |q'||latent|), a weight by 2 ds; v and the latent result are rounded once each,
        # and weights in both (2^-11): all of sum p |v|, but the latent result's rounding, which the projection carries on
        lat, n0, m0 = latent.double(), 0, 0
        other = torch.einsum("nhv,hdv->nhd", out2.double(), up_v.double())
        carried = 2.0 ** -11 * torch.einsum("nhv,hdv->nhd", out2.double().abs(), up_v.double().abs())
        for a, x in zip(add, lens):
            for h in range(H):
                if not a:
                    continue
                rows, keys = slice(n0, n0 + a), slice(m0, m0 + x)
                kk, vv = k[keys, h].double(), v[keys, h].double()
                seen = torch.arange(x, device="cuda")[None] <= torch.arange(x - a, x, device="cuda")[:, None]
                s = torch.where(seen, (q[rows, h, :128].double() @ kk.T + q[rows, h, 128:].double() @ rope[keys].double().T) * scale, -math.inf)
                ds = 2.0 ** -11 * scale * (q[rows, h, :128].double().abs() @ kk.abs().T + absorbed[rows, h, :V].double().abs() @ lat[keys].abs().T).amax(1)
                big = torch.softmax(s, 1) @ vv.abs()
                bound = 1.1 * ((4 * ds[:, None] + 4 * 2.0 ** -11 + 2.0 ** -14) * big + carried[rows, h]) + tol[rows, h]
                within(torch, other[rows, h], out[rows, h].double(), bound, "both forms")
            n0, m0 = n0 + a, m0 + x
