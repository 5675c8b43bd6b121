"""Calls of the prompt operators that their documentation allows and that lie at an edge (needs a GB300): workspaces used again,
one graph of several operators, values that are not finite in many units, rows behind the last request."""
from __future__ import annotations

import math

import numpy as np
import pytest

from tests import test_gpu_prompt as P
from tests.test_gpu_prompt import torch  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def test_one_workspace_for_calls_of_other_sizes(torch):  # noqa: F811
    """What an earlier call left in the workspace (joins, partial results, status) does not reach a later one."""
    cases = [P.prompt_case(torch, new, seq, H, dtype, 3) for new, seq, H, dtype in (
        ([7], [20000], 6, "bf16"), ([3, 200], [3, 200], 2, "f16"), ([600, 9], [4000, 9000], 16, "bf16"), ([1], [1], 1, "bf16"),
        ([20, 2, 300], [5000, 2, 400], 9, "f16"))]
    alone = [P.call_prompt(torch, c)[:2] for c in cases]
    ws = torch.full_like(P.call_prompt(torch, cases[0])[2], 0xff)
    for i in (0, 1, 2, 3, 4, 2, 0, 4, 1):
        out, lse, _, _ = P.call_prompt(torch, cases[i], ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])
    # calls in a row without a wait between them
    outs = [P.call_prompt(torch, cases[i], ws=ws)[:2] for i in (2, 0, 3, 4, 1)]
    torch.cuda.synchronize()
    for (out, lse), i in zip(outs, (2, 0, 3, 4, 1)):
        assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])


@pytest.mark.parametrize("new,seq,H", [([3, 2], [30000, 7], 5), ([256], [256], 7), ([768, 257], [768, 300], 3), ([1], [4000], 1024)])
def test_heads_in_pairs(torch, new, seq, H):  # noqa: F811
    """Last rows by two heads: odd numbers of heads, units cut into parts, many heads."""
    P.check_prompt(torch, P.prompt_case(torch, new, seq, H, "bf16", H))


@pytest.mark.parametrize("new,seq,H,dtype", [([300], [300], 456, "bf16"), ([200], [330], 700, "f16"), ([40, 513], [9000, 700], 12, "bf16")])
def test_values_that_are_not_finite_in_many_units(torch, new, seq, H, dtype):  # noqa: F811
    """Spoiled values in every second head, seen by the last rows: exactly those are spoiled, whatever else a CTA works on."""
    c = P.prompt_case(torch, new, seq, H, dtype, 9)
    ref, ref_lse, tol, tol_lse = P.reference(c) if H < 100 else (None,) * 4
    clean = P.call_prompt(torch, c)[:2]
    torch.cuda.synchronize()
    n0 = m0 = 0
    want = clean[0].double()
    for t, s in zip(new, seq):
        key = s - (t + 1) // 2
        c["v"][m0 + key, ::2, 5] = math.nan
        c["v"][m0 + key, ::2, 100] = math.inf
        first = n0 + max(0, key - (s - t))
        want[first:n0 + t, ::2, 5] = math.nan
        want[first:n0 + t, ::2, 100] = math.inf
        n0, m0 = n0 + t, m0 + s
    out, lse, ws, _ = P.call_prompt(torch, c)
    torch.cuda.synchronize()
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(out)[odd], torch.isnan(want)[odd]) and (out[odd & torch.isinf(want)] == math.inf).all()
    # the other columns: the taken-out value no longer adds to them (nor did it: columns are separate), so bit for bit
    assert torch.equal(out[~odd], clean[0][~odd]) and torch.equal(lse, clean[1])
    if ref is not None:
        P.within(torch, out.double()[~odd], ref[~odd], tol[~odd], "out")


def test_rows_behind_the_last_request(torch):  # noqa: F811
    """Queries behind the last request hold anything; keys behind it too."""
    c = P.prompt_case(torch, [100, 30], [400, 30], 3, "bf16", 2)
    good = P.call_prompt(torch, c)[:2]
    d = dict(c)
    d["q"] = torch.cat([c["q"], torch.full((200, 3, 192), math.nan, dtype=torch.bfloat16, device="cuda")])
    for k in ("k", "v"):
        d[k] = torch.cat([c[k], torch.full((300, 3, 128), math.nan, dtype=torch.bfloat16, device="cuda")])
    d["r"] = torch.cat([c["r"], torch.full((300, 64), math.inf, dtype=torch.bfloat16, device="cuda")])
    d["n"], d["m"] = 330, 730
    out, lse, ws, _ = P.call_prompt(torch, d)
    torch.cuda.synchronize()
    assert torch.equal(out[:130], good[0]) and torch.equal(lse[:130], good[1])
    assert (out[130:] == 7).all() and (lse[130:] == 7).all()


def test_one_graph_of_the_operators(torch):  # noqa: F811
    """Append, gather, rotation and attention captured once; replayed with new rows, positions and lengths."""
    import quantized_expert_ffn_bias_gb300 as coli
    t, page, H, B, room, rows = torch.bfloat16, 32, 4, 2, 400, 80
    W, V, ROT = P.W, P.V, P.ROT
    n_pages, max_pages = 30, 12
    kd = coli.coli_kv_desc(page, max_pages, n_pages, coli.COLI_X_BF16, page * W)
    rd = P.rope_desc(ROT, "half", "linear")
    freq = P.rope_table(torch, rd)
    g = P.gen(torch, 5)
    cache = torch.randn((n_pages, page, W), generator=g, device="cuda").to(t)
    table = P.ints(torch, np.random.default_rng(0).permutation(n_pages)[:B * max_pages].reshape(B, max_pages))
    seq, q_start = P.ints(torch, [200, 100]), P.ints(torch, [0, 50, 70])
    raw, q_raw = torch.zeros((rows, W), dtype=t, device="cuda"), torch.zeros((rows, H, 192), dtype=t, device="cuda")
    pos, slot = P.ints(torch, [0] * rows), P.ints(torch, [-1] * rows)
    kv = torch.randn((room, H, 256), generator=g, device="cuda").to(t)
    k_start, status = P.ints(torch, [0] * (B + 1)), P.ints(torch, [0])
    latent, rope = torch.zeros((room, V), dtype=t, device="cuda"), torch.zeros((room, ROT), dtype=t, device="cuda")
    q, out = torch.zeros_like(q_raw), torch.zeros((rows, H, 128), dtype=t, device="cuda")
    n_ws = coli.colibri_prompt_attention_workspace_size(B, rows, room, H)
    ws = torch.zeros(n_ws, dtype=torch.uint8, device="cuda")

    def step():
        st = torch.cuda.current_stream()
        coli.colibri_kv_append_rope(kd, rd, rows, q_start[B:], raw, W, None, 0.0, raw[:, V:], W, pos, freq, slot, cache, st)
        coli.colibri_kv_gather(kd, B, room, seq, table, cache, k_start, latent, V, rope, ROT, status, st)
        q.copy_(q_raw)
        coli.colibri_rope(rd, coli.COLI_X_BF16, rows, q_start[B:], H, pos, freq, q[..., 128:], H * 192, 192, q[..., 128:], H * 192, 192, st)
        coli.colibri_prompt_attention(coli.COLI_X_BF16, B, rows, room, H, 0.07, q, H * 192, 192, kv, H * 256, 256, rope, ROT,
                                      kv[..., 128:], H * 256, 256, q_start, k_start, out, None, ws, n_ws, st)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    free = np.setdiff1d(np.arange(n_pages), table.cpu().numpy())
    for i, (lens, new) in enumerate((([200, 100], [50, 20]), ([1, 384], [1, 79]), ([384, 0], [30, 0]), ([7, 9], [0, 9]))):
        raw.copy_(torch.randn(raw.shape, generator=g, device="cuda").to(t))
        q_raw.copy_(torch.randn(q_raw.shape, generator=g, device="cuda").to(t))
        pos.copy_(P.ints(torch, np.random.default_rng(i).integers(0, 5000, rows)))
        slot[page:] = -1                               # (one spare page: its rows once each)
        slot[:page] = P.ints(torch, free[0] * page + np.random.default_rng(i).permutation(page))
        seq.copy_(P.ints(torch, lens))
        q_start.copy_(P.ints(torch, np.concatenate([[0], np.cumsum(new)])))
        before = cache.clone()
        got = []
        for run in (graph.replay, step):
            cache.copy_(before)
            for x in (latent, rope, out, k_start):
                x.fill_(3)
            run()
            torch.cuda.synchronize()
            got.append([x.clone() for x in (cache, latent, rope, k_start, q, out)])
            assert coli.colibri_kv_check_status(ws) == 0 and int(status) == 0
        for a, b in zip(*got):
            assert torch.equal(a, b)
        assert (got[0][5][sum(new):] == 3).all()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype,N,H,dim,before,pad", [
    ("bf16", 70, 9, 64, 128, 4), ("bf16", 70, 9, 64, 128, 2), ("f16", 33, 5, 52, 2, 0), ("f16", 33, 5, 50, 2, 0), ("f32", 20, 3, 6, 2, 2),
    ("f32", 20, 3, 12, 0, 1), ("bf16", 1000, 1, 8, 0, 0), ("f16", 9, 128, 4, 4, 2), ("f32", 40, 2, 256, 0, 2), ("bf16", 3, 40, 254, 0, 0)])
def test_rotation_of_rows_of_any_alignment(torch, layout, dtype, N, H, dim, before, pad):  # noqa: F811
    """Vectors of 16, 8 and 4 bytes and single values, by what strides and the part's place allow; what lies beside is left."""
    import quantized_expert_ffn_bias_gb300 as coli
    from tests import prompt_ref as R
    t = P.dt(torch, dtype)
    d = P.rope_desc(dim, layout, "linear", 0.75)
    freq, g = P.rope_table(torch, d), P.gen(torch, N)
    wide = torch.randn((N, H * (before + dim) + pad), generator=g, device="cuda").to(t)
    x = wide[:, : H * (before + dim)].unflatten(1, (H, before + dim))[..., before:]
    pos = torch.randint(0, 100000, (N,), generator=g, device="cuda").to(torch.int32)
    ref, size = R.rotate(x.double(), pos, R.frequencies(dim, "linear"), layout, 0.75)
    tol = R.rotate_bound(ref, size, t) + size * (pos.double().view(-1, 1, 1) * 2.0 ** -51)
    again = wide.clone()
    y = again[:, : H * (before + dim)].unflatten(1, (H, before + dim))[..., before:]
    coli.colibri_rope(d, P.TYPES[dtype], N, None, H, pos, freq, y, y.stride(0), y.stride(1), y, y.stride(0), y.stride(1))
    torch.cuda.synchronize()
    P.within(torch, y, ref, tol, "in place")
    got = y.clone()
    y.copy_(x)
    assert torch.equal(again, wide)
    out = torch.full((H, N, dim + 2), 5.0, dtype=t, device="cuda")[..., 2:].transpose(0, 1)          # heads first, two values off
    coli.colibri_rope(d, P.TYPES[dtype], N, None, H, pos, freq, x, x.stride(0), x.stride(1), out, out.stride(0), out.stride(1))
    torch.cuda.synchronize()
    assert torch.equal(out, got)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_hand_overs_between_the_ctas_of_a_pair(torch, dtype):  # noqa: F811
    """Weights, rescaled sums and checked values of either CTA, many times over: rows within their bounds, every repetition the
    same bits.  The scores rise along the keys (references move in every tile), most tiles cross the diagonal, and some of their
    values are not finite."""
    c = P.prompt_case(torch, [500, 260, 7, 130], [700, 260, 3000, 1500], 10, dtype, 21)
    m0 = 0
    for s in c["seq"]:
        c["k"][m0:m0 + s, :, 0] = torch.linspace(0.0, 20.0, s, device="cuda")[:, None].to(c["k"].dtype)
        m0 += s
    c["q"][..., 0] = 4.0
    out, lse = P.check_prompt(torch, c)
    spoiled = dict(c, v=c["v"].clone())
    spoiled["v"][[650, 900], ::3, 9] = math.inf
    spoiled["v"][[650, 900], 1::3, 70] = -math.inf
    odd = P.call_prompt(torch, spoiled)[0]
    ws = torch.zeros_like(P.call_prompt(torch, c)[2])
    for _ in range(60):
        got = P.call_prompt(torch, c, ws=ws)[:2]
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        assert torch.equal(P.call_prompt(torch, spoiled, ws=ws)[0], odd)
    # rows of requests 0 and 1 from the spoiled keys on (their own rows 450 and 200), in the heads and columns that were spoiled
    want = out.clone()
    for head, column, what in ((0, 9, math.inf), (1, 70, -math.inf)):
        want[450:500, head::3, column] = what
        want[700:760, head::3, column] = what
    assert torch.equal(odd, want)


@pytest.mark.parametrize("new,seq,dtype", [([3], [200], "bf16"), ([3], [20000], "bf16"), ([2, 300], [9000, 12000], "f16")])
@pytest.mark.parametrize("far", [0.0, 0.5])
def test_values_that_are_not_finite_behind_weights_of_nothing(torch, new, seq, dtype, far):  # noqa: F811
    """A stretch of keys scores some 300 below the others (weights below fp32's range): its infinities and NaN still reach the rows
    that see them, whether the keys are cut into parts or not, and nothing else changes."""
    c = P.prompt_case(torch, new, seq, 4, dtype, 31)
    c["q"][..., 0] = 64.0
    c["k"][..., 0] = 0.0
    marks, m0 = [], 0
    for b, s in enumerate(seq):
        first, last = int(far * s), int(far * s) + s // 4
        c["k"][m0 + first:m0 + last, :, 0] = -64.0       # 64 * 64 / sqrt(192) = 295
        marks.append([(m0 + (first + last) // 2, b, math.inf), (m0 + last - 1, 2, math.nan)])
        m0 += s
    ref, ref_lse, tol, tol_lse = P.reference(c)          # (before the values are spoiled: theirs weigh nothing)
    odd, n0 = torch.zeros_like(ref, dtype=torch.bool), 0
    for t, two in zip(new, marks):
        for key, h, what in two:
            c["v"][key, h, 11 + h] = what
            odd[n0:n0 + t, h, 11 + h] = True             # (the stretch ends before the new tokens)
        n0 += t
    out, lse, ws, _ = P.call_prompt(torch, c)
    torch.cuda.synchronize()
    assert not torch.isfinite(out[odd]).any()
    P.within(torch, out[~odd], ref[~odd], tol[~odd], "the others")
    P.within(torch, lse, ref_lse, tol_lse, "lse")


@pytest.mark.parametrize("new,seq", [([5], [300]), ([3], [20000]), ([10], [4]), ([600], [700]), ([2, 270], [9000, 11000])])
def test_rows_whose_scores_are_all_minus_infinity(torch, new, seq):  # noqa: F811
    """The softmax of minus infinities alone is NaN, its sum's log minus infinity; one finite score takes all the weight; rows
    without keys stay 0."""
    c = P.prompt_case(torch, new, seq, 3, "bf16", 32)
    c["q"][..., 0] = 1.0
    c["k"][..., 0] = -math.inf
    alone = P.call_prompt(torch, c)[:2]
    m0, finite = 0, []
    for t, s in zip(new, seq):
        finite.append(max(0, s - t // 2 - 1))            # rows before it see no finite score
        c["k"][m0 + finite[-1], :, 0] = 0.0
        m0 += s
    one = P.call_prompt(torch, c)[:2]
    torch.cuda.synchronize()
    n0 = m0 = 0
    for t, s, key in zip(new, seq, finite):
        last = torch.arange(t, device="cuda") + (s - t)  # the last key that a row sees
        for (out, lse), some in ((alone, torch.zeros_like(last, dtype=torch.bool)), (one, last >= key)):
            o, z = out[n0:n0 + t], lse[n0:n0 + t]
            assert (o[last < 0] == 0).all() and (z[last < 0] == -math.inf).all()
            none = (last >= 0) & ~some
            assert torch.isnan(o[none]).all() and (z[none] == -math.inf).all()
            # its one weight w is rounded to the type for the product and not in the sum: w (1 + d) v / w with |d| <= eps / 2, a
            # reciprocal and a product in fp32 (2^-22), the result's rounding: (1 + eps / 2)^2 (1 + 2^-22) - 1 < 1.01 eps
            v = c["v"][m0 + key].double().expand(int(some.sum()), -1, -1)
            P.within(torch, o[some], v, 1.01 * torch.finfo(torch.bfloat16).eps * v.abs() + 2.0 ** -133, "out")
            q, k = c["q"][n0:n0 + t][some].double(), c["k"][m0 + key].double()
            score = (torch.einsum("nhd,hd->nh", q[..., :128], k) + q[..., 128:] @ c["r"][m0 + key].double()) * c["scale"]
            # 192 exact products summed in fp32 (2^-23 each of their magnitudes' sum), the scale and the log's few roundings
            size = (torch.einsum("nhd,hd->nh", q[..., :128].abs(), k.abs()) + q[..., 128:].abs() @ c["r"][m0 + key].double().abs()) * c["scale"]
            P.within(torch, z[some], score, 200 * 2.0 ** -23 * size + 2.0 ** -21 * (score.abs() + 1), "lse")
        n0, m0 = n0 + t, m0 + s


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("count", [-2**31, -2**31 + 40, -3, 0, 2**31 - 1])
def test_rotation_of_any_count(torch, layout, count):  # noqa: F811
    """Rows from the count on are left, whatever the count: below 0 it leaves all of them, in every block of rows."""
    import quantized_expert_ffn_bias_gb300 as coli
    d = P.rope_desc(64, layout)
    x = torch.randn((700, 2, 64), generator=P.gen(torch, 1), device="cuda").bfloat16()
    pos, freq = torch.arange(700, dtype=torch.int32, device="cuda"), P.rope_table(torch, d)
    want, out = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    if count > 0:
        coli.colibri_rope(d, 0, 700, None, 2, pos, freq, x, 128, 64, want, 128, 64)
    coli.colibri_rope(d, 0, 700, P.ints(torch, [count]), 2, pos, freq, x, 128, 64, out, 128, 64)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and (out[600] == 5.0).all() == (count <= 0)


@pytest.mark.parametrize("eps", [1e-38, 1e30, 1e36, 3.4e38])
def test_norm_with_any_eps(torch, eps):  # noqa: F811
    """An eps that decides, up to fp32's largest: rows far smaller than its root stay what they are over it, rows that overflow
    in their squares are normed."""
    import quantized_expert_ffn_bias_gb300 as coli
    from tests import prompt_ref as R
    eps = float(torch.tensor(eps, dtype=torch.float32))
    sizes = torch.tensor([1e-38, 1e-20, 1e-18, 1e-3, 1.0, 1e3, 1e15, 1e17, 5e18, 1e19, 2e25, 3e38], device="cuda", dtype=torch.float64)
    n, t = len(sizes), torch.bfloat16
    c = P.append_case(torch, "bf16", n, 16, "half", True, 3)
    unit = torch.rand((n, P.V), generator=P.gen(torch, 4), device="cuda").double() * 0.9 + 0.1
    c["latent"] = (unit * sizes[:, None]).float().to(t)
    rd = P.rope_desc(64, "half")
    cache = c["cache"].clone()
    P.call_append(c, coli.coli_kv_desc(16, 1, c["n_pages"], 0, 16 * P.W), rd, P.rope_table(torch, rd), n, None, eps, cache)
    torch.cuda.synchronize()
    got = cache.view(-1, P.W)[c["slot"].long(), :P.V]
    ref = R.norm(c["latent"].double(), c["gain"].double(), eps)
    # (what is below fp32's normal range before the gain may lose all of its bits)
    P.within(torch, got, ref, R.norm_bound(ref, t) + 2.0 ** -126 * c["gain"].double().abs(), "latent")
