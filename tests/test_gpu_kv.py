"""The paged compressed cache on the GPU (needs a GB300): bookkeeping and appending against plain forms (equal), attention
against the 64-bit form within its error bounds, and a run of them together with the key selection and a layer forward."""
from __future__ import annotations

import numpy as np
import pytest

from tests import serving_ref as R

pytestmark = pytest.mark.gpu

W, V = R.WIDTH, R.VALUE


@pytest.fixture(scope="module")
def torch_cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_expert_ffn_bias_gb300 as coli
    coli.build()
    return torch


def ints(torch, a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


# ---------------------------------------------------------------- bookkeeping


def call_step(torch, page, max_pages, n_pages, n_tokens, new, seq, held, table, free, count, in_place=False, stream=None):
    import quantized_expert_ffn_bias_gb300 as coli
    B = len(new)
    d = coli.coli_kv_desc(page, max_pages, n_pages, 0, page * W)
    t = dict(new=ints(torch, new), seq=ints(torch, seq), held=ints(torch, held), table=ints(torch, table),
             free=ints(torch, free), count=ints(torch, [count]))
    if in_place:
        t.update(seq_out=t["seq"], held_out=t["held"], count_out=t["count"])
    else:
        t.update(seq_out=ints(torch, [-9] * B), held_out=ints(torch, [-9] * B), count_out=ints(torch, [-9]))
    t.update(q_start=ints(torch, [-9] * (B + 1)), position=ints(torch, [-9] * (n_tokens + 5)),
             slot=ints(torch, [-9] * (n_tokens + 5)), status=ints(torch, [0]))
    coli.colibri_kv_step(d, B, n_tokens, t["new"], t["seq"], t["held"], t["table"], t["free"], t["count"], t["seq_out"],
                         t["held_out"], t["count_out"], t["q_start"], t["position"], t["slot"], t["status"],
                         stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in t.items()}


def check_step(torch, *a, **kw):
    for in_place in (False, True):
        got = call_step(torch, *a, in_place=in_place, **kw)
        page, max_pages, n_pages, n_tokens, new, seq, held, table, free, count = a
        ref = R.step(page, max_pages, n_pages, n_tokens, list(map(int, new)), list(map(int, seq)), list(map(int, held)),
                     np.asarray(table, np.int32), np.asarray(free, np.int32), int(count))
        for k in ("seq_out", "held_out", "q_start", "table", "free"):
            np.testing.assert_array_equal(got[k], ref[k], err_msg=k)
        assert got["count_out"][0] == ref["count_out"]
        assert got["status"][0] == ref["status"]
        n = len(ref["position"])
        np.testing.assert_array_equal(got["position"][:n], ref["position"])
        np.testing.assert_array_equal(got["slot"][:n], ref["slot"])
        assert (got["position"][n:] == -9).all() and (got["slot"][n:] == -9).all(), "rows behind the last request"
    return ref


def make_state(rng, B, page, past, extra_pages=20, spare_cols=2, hold_more=True):
    seq = rng.integers(0, past + 1, B)
    held = -(-seq // page) + (rng.integers(0, 2, B) if hold_more else 0)
    max_pages = int(held.max()) + spare_cols + -(-40 // page)
    n_pages = int(held.sum()) + extra_pages
    order = rng.permutation(n_pages)
    table = np.full((B, max_pages), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(n_pages, -1, np.int32)
    free[:n_pages - at] = order[at:]
    return seq, held, max_pages, n_pages, table, free, n_pages - at


@pytest.mark.parametrize("B,page,past,new_hi,extra", [
    (1, 1, 0, 1, 4), (1, 64, 0, 3, 4), (3, 16, 50, 40, 20), (64, 64, 3000, 4, 100), (1000, 16, 200, 9, 1200),
    (1025, 48, 500, 2, 400), (8192, 64, 300, 3, 5000)])
def test_step_matches_plain(torch_cuda, B, page, past, new_hi, extra):
    rng = np.random.default_rng(B + page)
    seq, held, mp, n, table, free, count = make_state(rng, B, page, past, extra)
    new = rng.integers(0, new_hi + 1, B)
    if B > 2:
        new[rng.random(B) < 0.1] = -1
    check_step(torch_cuda, page, mp, n, int(new.clip(0).sum()) + 3, new, seq, held, table, free, count)


def test_step_refuses_what_does_not_fit(torch_cuda):
    rng = np.random.default_rng(1)
    B, page = 300, 16
    seq, held, mp, n, table, free, count = make_state(rng, B, page, 200, extra_pages=60, hold_more=False)
    new = rng.integers(0, 30, B)
    new[::13] = -1
    ref = check_step(torch_cuda, page, mp, n, int(new.clip(0).sum()), new, seq, held, table, free, count)   # pages run out
    assert ref["status"] == R.NO_PAGES
    ref = check_step(torch_cuda, page, mp, n, 900, np.minimum(new, 3 * (seq % page > 0)), seq, held, table, free, count)
    ref = check_step(torch_cuda, page, mp, n, 200, new, seq, held, table, free, count)                        # rows run out
    assert ref["status"] & R.TOKENS
    bad_seq, bad_held, bad_new = seq.copy(), held.copy(), new.copy()
    bad_seq[3], bad_held[5], bad_held[8], bad_new[11] = -4, -1, mp + 1, mp * page + 1
    bad_held[13] = mp + 7                                                                                      # finished, not valid
    bad_seq[20] = held[20] * page + 1
    ref = check_step(torch_cuda, page, mp, n, int(new.clip(0).sum()), bad_new, bad_seq, bad_held, table, free, count)
    assert ref["status"] & R.TABLE_FULL


def test_step_bad_pages_and_counts(torch_cuda):
    rng = np.random.default_rng(2)
    B, page = 40, 8
    seq, held, mp, n, table, free, count = make_state(rng, B, page, 100, 60, hold_more=False)
    seq = np.maximum(seq, 1)
    held = -(-seq // page)
    table = np.where(np.arange(mp)[None] < held[:, None], np.where(table < 0, 0, table), -1).astype(np.int32)
    table[4, held[4] - 1], table[9, held[9] - 1] = -1, n
    seq[4], seq[9] = held[4] * page - 1, held[9] * page - 1
    new = np.full(B, 1)
    ref = check_step(torch_cuda, page, mp, n, B, new, seq, held, table, free, count)
    assert ref["status"] == R.BAD_PAGE and (ref["slot"] == -1).sum() >= 2
    for wrong in (-3, n + 5):
        check_step(torch_cuda, page, mp, n, B, np.zeros(B, int), seq, held, table, free, wrong)
    new[::2] = -1
    check_step(torch_cuda, page, mp, n, B, new, seq, held, table, free, n - 1)     # more pages come back than the stack holds


def test_step_empty_batches(torch_cuda):
    rng = np.random.default_rng(3)
    seq, held, mp, n, table, free, count = make_state(rng, 5, 16, 60)
    check_step(torch_cuda, 16, mp, n, 0, np.zeros(5, int), seq, held, table, free, count)
    check_step(torch_cuda, 16, mp, n, 4, np.full(5, -1), seq, held, table, free, count)


# ---------------------------------------------------------------- append


@pytest.mark.parametrize("n,page,dtype,pad,gap", [(1, 1, "bf16", 0, 0), (7, 48, "f16", 8, 0), (300, 64, "bf16", 64, 2),
                                                  (20000, 16, "bf16", 0, 1)])
def test_append_copies_rows(torch_cuda, n, page, dtype, pad, gap):
    torch = torch_cuda
    import quantized_expert_ffn_bias_gb300 as coli
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    n_pages, stride = -(-n // page) + 3, (page + gap) * W
    cache = torch.randint(-30000, 30000, (n_pages, stride), generator=g, device="cuda", dtype=torch.int16)
    lat = torch.randint(-30000, 30000, (n + 2, V + pad), generator=g, device="cuda", dtype=torch.int16)
    rope = torch.randint(-30000, 30000, (n + 2, 64 + pad), generator=g, device="cuda", dtype=torch.int16)
    slot = torch.randperm(n_pages * page, generator=g, device="cuda")[:n + 2].to(torch.int32)
    valid = n if n < 5 else n - 2
    if n > 5:
        slot[1], slot[3] = -1, n_pages * page
    want = cache.clone()
    for i in range(valid):
        s = int(slot[i]) if n < 1000 else None
        if s is not None and 0 <= s < n_pages * page:
            want[s // page, (s % page) * W:(s % page) * W + V] = lat[i, :V]
            want[s // page, (s % page) * W + V:(s % page + 1) * W] = rope[i, :64]
    if n >= 1000:
        ok = (slot[:valid] >= 0) & (slot[:valid] < n_pages * page)
        s = slot[:valid][ok].long()
        rows = want.view(n_pages, page + gap, W)
        rows[s // page, s % page] = torch.cat([lat[:valid, :V], rope[:valid, :64]], 1)[ok]
    d = coli.coli_kv_desc(page, 1, n_pages, {"bf16": 0, "f16": 2}[dtype], stride)
    coli.colibri_kv_append(d, n, ints(torch, [valid]), lat, V + pad, rope, 64 + pad, slot, cache, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(cache, want)
    coli.colibri_kv_append(d, 0, None, None, 0, None, 0, None, None, None)
    coli.colibri_kv_append(d, n, ints(torch, [-5]), lat, V + pad, rope, 64 + pad, slot, cache, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(cache, want), "a negative count writes nothing"


# ---------------------------------------------------------------- attention


class Batch:
    """Requests with lengths (tokens in the cache, new tokens), a cache of random rows, block tables in random order."""

    def __init__(self, torch, lens, new, H, page, dtype="bf16", seed=0, gap=0, spare_rows=0, qpad=0, q_order="nhw",
                 qscale=1.5):
        self.torch, self.lens, self.new, self.H, self.page, self.dtype = torch, list(lens), list(new), H, page, dtype
        self.dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
        rng = np.random.default_rng(seed)
        held = [R.pages_of(v, page) for v in lens]
        self.n_pages = sum(held) + 3
        self.max_pages = max(held + [1]) + 1
        self.stride = (page + gap) * W
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = order[at:at + h]
            at += h
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.N = int(self.q_start[-1]) + spare_rows
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        self.cache = torch.randn((self.n_pages, self.stride), generator=g, device="cuda").to(self.dt)
        shape = {"nhw": (self.N, H, W + qpad), "hnw": (H, self.N, W + qpad)}[q_order]
        q = (torch.randn(shape, generator=g, device="cuda") * qscale).to(self.dt)
        self.q = (q if q_order == "nhw" else q.transpose(0, 1))[:, :, :W]
        self.scale = W ** -0.5

    def run(self, sel=None, lse=True, ws=None, stream=None, fill=3.0, status=0):
        torch = self.torch
        import quantized_expert_ffn_bias_gb300 as coli
        d = coli.coli_kv_desc(self.page, self.max_pages, self.n_pages, {"bf16": 0, "f16": 2}[self.dtype], self.stride)
        B = len(self.lens)
        n = coli.colibri_kv_attention_workspace_size(B, self.N, self.H)
        if ws is None:
            ws = torch.randint(0, 255, (n,), dtype=torch.uint8, device="cuda")
        out = torch.full((self.N, self.H, V), fill, dtype=self.dt, device="cuda")
        z = torch.full((self.N, self.H), fill, device="cuda") if lse else None
        st = stream or torch.cuda.current_stream()
        sd = ints(torch, sel) if sel is not None else None
        args = [ints(torch, self.table), ints(torch, self.q_start), ints(torch, self.lens)]
        torch.cuda.synchronize()
        coli.colibri_kv_attention(d, B, self.N, self.H, self.scale, self.q, self.q.stride(0), self.q.stride(1), self.cache,
                                  *args, sd, sd.shape[1] if sd is not None else 0, out, z, ws, n, st)
        torch.cuda.synchronize()
        assert coli.colibri_kv_check_status(ws, st) == status
        return out, z

    def check(self, sel=None, **kw):
        torch = self.torch
        out, z = self.run(sel=sel, **kw)
        flat = self.cache.double().cpu().numpy().ravel()
        cache = R.Cache(flat, self.page, self.stride)
        info = torch.finfo(self.dt)
        ref, lse, tol, tol_lse, done = R.attention(
            self.q.double().cpu().numpy(), cache, self.table, self.q_start, self.lens, self.scale, info.eps, sel=sel,
            tiny=float(info.smallest_normal) * info.eps)
        o = out.double().cpu().numpy()
        err = np.abs(o - ref)
        bad = ~(err <= tol)
        bad[~done] = False
        assert not bad.any(), f"{bad.sum()} of {bad.size} beyond the bound, first {np.argwhere(bad)[:3].tolist()}: " \
                              f"{o[bad][:3]} vs {ref[bad][:3]}, bound {tol[bad][:3]}"
        assert (o[~done] == 3.0).all(), "rows outside the requests"
        if z is not None:
            zz = z.double().cpu().numpy()
            none = np.isneginf(lse) & done[:, None]
            assert np.isneginf(zz[none]).all() and (o[none] == 0).all(), "rows that see no key"
            fin = ~np.isneginf(lse)
            assert (np.abs(zz[fin] - lse[fin]) <= tol_lse[fin]).all()
            assert (zz[~done] == 3.0).all()
        return out, z


def selected(rng, lens, new, topk, frac=1.0):
    """topk distinct visible keys of each token (fewer where it sees fewer), ascending, -1 behind."""
    rows = []
    for ln, T in zip(lens, new):
        for t in range(T):
            seen = ln - T + t + 1
            m = min(int(topk * frac), seen)
            s = np.sort(rng.choice(seen, m, replace=False)) if m > 0 else np.array([], int)
            rows.append(np.concatenate([s, np.full(topk - m, -1)]))
    return np.array(rows, np.int32)


DENSE = [
    # lens, new, H, page, more
    ([1], [1], 1, 1, {}),
    ([5], [5], 16, 16, dict(dtype="f16")),
    ([128], [1], 64, 64, {}),
    ([129, 127, 1], [1, 2, 1], 64, 64, {}),
    ([300, 40, 700], [3, 3, 3], 64, 48, dict(dtype="f16", gap=2)),
    ([513, 0, 77, 200], [1, 0, 5, 0], 128, 16, dict(spare_rows=4)),
    ([1000], [70], 16, 7, dict(qpad=64)),
    ([260, 131], [130, 131], 3, 32, dict(q_order="hnw")),
    ([400], [9], 65, 128, {}),
    ([2500], [1], 8, 64, {}),
    ([90, 95], [2, 1], 96, 256, dict(qscale=12.0)),
]


@pytest.mark.parametrize("case", range(len(DENSE)))
def test_attention_dense(torch_cuda, case):
    lens, new, H, page, kw = DENSE[case]
    Batch(torch_cuda, lens, new, H, page, seed=case, **kw).check()


@pytest.mark.parametrize("lens,new,H,topk,frac", [
    ([300], [1], 64, 64, 1.0), ([700, 90], [3, 2], 64, 256, 1.0), ([1500], [4], 16, 500, 0.7), ([600, 3], [2, 3], 128, 130, 1.0),
    ([2200], [2], 64, 2048, 1.0)])
def test_attention_selected_keys(torch_cuda, lens, new, H, topk, frac):
    rng = np.random.default_rng(topk)
    b = Batch(torch_cuda, lens, new, H, 64, seed=topk)
    b.check(sel=selected(rng, lens, new, topk, frac))


def test_attention_selected_in_any_order_twice_beyond_and_none(torch_cuda):
    """Entries in any order, one twice, some beyond the position or negative; a token with no entry at all; the first
    tile of a list without an entry."""
    rng = np.random.default_rng(4)
    lens, new = [500, 300], [3, 2]
    b = Batch(torch_cuda, lens, new, 64, 32, seed=4)
    sel = selected(rng, lens, new, 300)
    sel[0] = rng.permutation(sel[0])
    sel[1, 10], sel[1, 20:30], sel[1, 40] = sel[1, 11], 499, -77          # token 1 is at position 498
    sel[2] = -1
    sel[3, :200] = -1
    sel[4, 100:] = 299
    b.check(sel=sel)


def test_attention_references_rise(torch_cuda):
    """Keys whose scores grow along the sequence (every tile raises the references), and the reverse order."""
    torch = torch_cuda
    for sign in (1.0, -1.0):
        b = Batch(torch, [1300], [2], 16, 64, seed=6)
        grow = torch.linspace(0, 3, 1300, device="cuda") if sign > 0 else torch.linspace(3, 0, 1300, device="cuda")
        rows = b.cache.view(b.n_pages, 64, W)
        direction = b.q[0, 0].float()
        for j in range(1300):
            pg = int(b.table[0, j // 64])
            rows[pg, j % 64] = (rows[pg, j % 64].float() + direction * grow[j]).to(b.dt)
        b.check()


def test_attention_row_without_keys(torch_cuda):
    """More new tokens than cached ones (a request whose rows were not appended): the rows before the first key get 0."""
    b = Batch(torch_cuda, [64, 2], [1, 5], 64, 16, seed=8)
    b.check()
    b = Batch(torch_cuda, [0], [2], 16, 16, seed=9)
    b.check()


def test_attention_ignores_values_of_unseen_keys(torch_cuda):
    """Infinities and NaN in rows a token does not see -- behind the last key, in other pages, in later new tokens -- do
    not reach it; the tokens that see such a row get a result that is not finite."""
    torch = torch_cuda
    lens, new = [200, 131], [4, 3]
    b = Batch(torch, lens, new, 64, 64, seed=10)
    clean, zc = b.run()
    rows = b.cache.view(b.n_pages, 64, W)
    used = np.zeros((b.n_pages, 64), bool)
    for i, ln in enumerate(lens):
        for j in range(ln):
            used[b.table[i, j // 64], j % 64] = True
    junk = torch.from_numpy(~used).cuda()
    for v in (float("nan"), float("inf"), float("-inf"), torch.finfo(b.dt).max, torch.finfo(b.dt).min):
        rows[junk] = v
        out, z = b.run()
        assert torch.equal(out, clean) and torch.equal(z, zc)
    for v in (float("nan"), float("inf")):
        pg = int(b.table[0, 199 // 64])
        rows[pg, 199 % 64, :] = v                                # seen by the last token of request 0 alone
        out, z = b.run()
        assert torch.equal(out[:3], clean[:3]) and torch.equal(out[4:], clean[4:])
        assert not torch.isfinite(out[3]).any()


def test_attention_unseen_keys_in_selection(torch_cuda):
    torch = torch_cuda
    b = Batch(torch, [300], [2], 64, 64, seed=12)
    sel = selected(np.random.default_rng(1), [300], [2], 100, 0.6)
    clean, _ = b.run(sel=sel)
    rows = b.cache.view(b.n_pages, 64, W)
    named = set(sel[sel >= 0].tolist())
    for j in range(300):
        if j not in named:
            rows[int(b.table[0, j // 64]), j % 64] = float("nan")
    for pg in set(range(b.n_pages)) - set(b.table[0][b.table[0] >= 0].tolist()):
        rows[pg] = float("inf")
    out, _ = b.run(sel=sel)
    assert torch.equal(out, clean)


def test_attention_query_with_nan_stays_in_its_row(torch_cuda):
    torch = torch_cuda
    b = Batch(torch, [200], [3], 64, 64, seed=13)
    clean, _ = b.run()
    b.q[1, 7, 100] = float("nan")
    out, _ = b.run()
    keep = torch.ones((3, 64), dtype=torch.bool)
    keep[1, 7] = False
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[1, 7]).all()


def test_attention_reports_bad_pages(torch_cuda):
    b = Batch(torch_cuda, [300, 100], [1, 2], 64, 32, seed=14)
    b.table[0, 3], b.table[0, 5] = -1, b.n_pages
    b.check(status=R.BAD_PAGE)
    b = Batch(torch_cuda, [256, 100], [1, 2], 64, 32, seed=16)      # a request longer than its row of the table
    b.table, b.max_pages = np.ascontiguousarray(b.table[:, :4]), 4
    b.check(status=R.BAD_PAGE)


def test_attention_refuses_a_wrong_q_start(torch_cuda):
    """Not ascending: nothing is written and the status says so.  Beyond the batch: the rows that exist are computed."""
    torch = torch_cuda
    b = Batch(torch_cuda, [300, 100, 50], [2, 2, 2], 64, 32, seed=15)
    b.q_start = np.array([0, 4, 2, 6], np.int32)
    out, z = b.run(status=R.TOKENS)
    assert (out == 3.0).all() and (z == 3.0).all()
    b.q_start = np.array([0, 2, 4, 1 << 30], np.int32)
    out, _ = b.run()
    assert torch.isfinite(out).all()


def test_attention_long_context_and_splits(torch_cuda):
    """One unit cut over every SM, uneven units cut at odd places: against the sum over thirds of the keys in 64 bits."""
    torch = torch_cuda
    for lens, new, H, page in (([30011], [1], 64, 64), ([9000, 300, 7001, 25, 4100], [3, 1, 2, 1, 4], 16, 128),
                               ([3000] * 40, [1] * 40, 8, 64)):
        b = Batch(torch, lens, new, H, page, seed=len(lens))
        b.check()


@pytest.mark.parametrize("scale", [0.0, -0.04, 1e-6])
def test_attention_any_finite_scale(torch_cuda, scale):
    b = Batch(torch_cuda, [300, 77], [3, 2], 64, 64, seed=51)
    b.scale = scale
    b.check()
    b.check(sel=selected(np.random.default_rng(3), [300, 77], [3, 2], 90, 0.8))


def test_attention_many_requests(torch_cuda):
    """The most requests a call takes, a few keys each."""
    rng = np.random.default_rng(50)
    lens = rng.integers(0, 9, 8192)
    Batch(torch_cuda, lens, np.minimum(lens, rng.integers(0, 3, 8192)), 2, 16, seed=50).check()


def test_attention_gangs(torch_cuda):
    """Keys beyond what stays in L2, several row tiles over the same keys: gangs of CTAs walk them together, some with idle
    members (requests of one, two and four tokens among those of three)."""
    rng = np.random.default_rng(60)
    new = [3, 1, 3, 2, 3, 3, 4, 3, 3, 3]
    b = Batch(torch_cuda, rng.integers(5500, 9000, 10), new, 64, 64, seed=60)
    b.check()
    b = Batch(torch_cuda, rng.integers(5500, 9000, 8), [1] * 8, 160, 128, seed=61, dtype="f16")
    b.check()


def test_attention_gangs_over_selected_keys(torch_cuda):
    rng = np.random.default_rng(62)
    lens, new = list(rng.integers(3000, 5000, 10)), [3] * 10
    b = Batch(torch_cuda, lens, new, 128, 64, seed=62)
    b.check(sel=selected(rng, lens, new, 2048))


def test_attention_does_not_depend_on_timing_or_workspace(torch_cuda):
    torch = torch_cuda
    b = Batch(torch, [5000, 800], [3, 2], 64, 64, seed=20)
    first, z = b.run()
    for _ in range(3):
        out, z2 = b.run()
        assert torch.equal(out, first) and torch.equal(z, z2)
    assert torch.equal(b.run(lse=False)[0], first)


def test_attention_rows_beyond_32_bit_offsets(torch_cuda):
    """A cache of more than 2^32 bytes and 2^31 elements: the last pages' rows are the right ones."""
    torch = torch_cuda
    import quantized_expert_ffn_bias_gb300 as coli
    page, n_pages = 64, (1 << 31) // (64 * W) + 40
    cache = torch.zeros((n_pages, page * W), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    small = Batch(torch, [300], [2], 64, page, seed=21)
    high = small.table.copy()
    for i in range(R.pages_of(300, page)):
        high[0, i] = n_pages - 1 - 3 * i
        cache[n_pages - 1 - 3 * i] = small.cache[int(small.table[0, i])]
    want, _ = small.run()
    small.cache, small.table, small.n_pages = cache, high, n_pages
    got, _ = small.run()
    assert torch.equal(got, want)
    # and append reaches them
    d = coli.coli_kv_desc(page, 1, n_pages, 0, page * W)
    row = torch.randn((1, W), generator=g, device="cuda").to(torch.bfloat16)
    coli.colibri_kv_append(d, 1, None, row, W, row[:, V:], W, ints(torch, [n_pages * page - 1]), cache,
                           torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(cache[-1, -W:], row[0])


def test_attention_two_streams_and_a_graph(torch_cuda):
    torch = torch_cuda
    import quantized_expert_ffn_bias_gb300 as coli
    a = Batch(torch, [4000, 100], [2, 1], 64, 64, seed=30)
    b = Batch(torch, [900] * 9, [3] * 9, 32, 64, seed=31, dtype="f16")
    wa, wb = a.run()[0], b.run()[0]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held = []
    for x, s in ((a, streams[0]), (b, streams[1])):
        d = coli.coli_kv_desc(x.page, x.max_pages, x.n_pages, {"bf16": 0, "f16": 2}[x.dtype], x.stride)
        n = coli.colibri_kv_attention_workspace_size(len(x.lens), x.N, x.H)
        held.append((x, s, d, n, torch.empty(n, dtype=torch.uint8, device="cuda"), ints(torch, x.table), ints(torch, x.q_start),
                     ints(torch, x.lens), torch.zeros((x.N, x.H, V), dtype=x.dt, device="cuda")))
    torch.cuda.synchronize()

    def call(h, st):
        x, _, d, n, ws, tb, qs, ln, out = h
        coli.colibri_kv_attention(d, len(x.lens), x.N, x.H, x.scale, x.q, x.q.stride(0), x.q.stride(1), x.cache, tb, qs, ln,
                                  None, 0, out, None, ws, n, st)
    for _ in range(10):
        for h in held:
            call(h, h[1])
    torch.cuda.synchronize()
    assert torch.equal(held[0][-1], wa) and torch.equal(held[1][-1], wb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(held[0], torch.cuda.current_stream())
        call(held[1], torch.cuda.current_stream())
    held[0][-1].zero_()
    held[1][-1].zero_()
    # the graph reads lengths on the GPU: a shorter request in the same buffers
    a.lens = [3500, 90]
    held[0][7].copy_(ints(torch, a.lens))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0][-1], a.run()[0]) and torch.equal(held[1][-1], wb)


# ---------------------------------------------------------------- together


def test_serving_step_together(torch_cuda):
    """Steps of a few requests as they would be served: bookkeeping, appending, key selection, attention over the selected
    keys, and a layer forward with group-limited routing -- chunk, then verify steps with drafts taken back, a finished
    request.  The cache always holds what the plain form says, the attention is the 64-bit form's."""
    torch = torch_cuda
    import harness as H
    import quantized_expert_ffn_bias_gb300 as coli
    from harness.device import DeviceLayer
    rng = np.random.default_rng(40)
    page, B, heads, topk = 32, 3, 64, 128
    mp, n_pages, n_tok = 24, 40, 400
    d = coli.coli_kv_desc(page, mp, n_pages, 0, page * W)
    st = torch.cuda.current_stream()
    cache = torch.full((n_pages, page * W), float("nan"), dtype=torch.bfloat16, device="cuda")
    table, free, count = np.full((B, mp), -1, np.int32), rng.permutation(n_pages).astype(np.int32), n_pages
    seq, held = np.zeros(B, int), np.zeros(B, int)
    t = dict(table=ints(torch, table), free=ints(torch, free), count=ints(torch, [count]), seq=ints(torch, seq),
             held=ints(torch, held), q_start=ints(torch, [0] * (B + 1)), position=ints(torch, [0] * n_tok),
             slot=ints(torch, [0] * n_tok), status=ints(torch, [0]))
    layer = H.gen_layer(72, 0, d=512, F=256, E=32, k=4, rho=2.5, qtype=H.Q_INT4_G128, bias="uniform:0.1")
    dl = DeviceLayer(layer, 512)
    dl.plan.set_route(coli.coli_route_desc(32, 4, 0, 4, 2, 0, 1, 2.5))
    up = torch.randn((heads * V, 512), device="cuda") / (heads * V) ** 0.5
    n_ws = coli.colibri_kv_attention_workspace_size(B, n_tok, heads)
    ws = torch.empty(n_ws, dtype=torch.uint8, device="cuda")
    ix_ws = torch.empty(coli.colibri_indexer_workspace_size(n_tok, 1024), dtype=torch.uint8, device="cuda")
    keys_all = [np.zeros((0, W)) for _ in range(B)]             # what each request's cache should hold
    ix_keys = [torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda") for _ in range(B)]
    back = [0, 0, 0]
    for step, new in enumerate(([200, 90, 1], [3, 3, 3], [3, -1, 3], [3, 50, 3])):
        seq = np.maximum(seq - back, 0)                          # drafts taken back
        t["seq"].copy_(ints(torch, seq))
        for b in range(B):
            keys_all[b], ix_keys[b] = keys_all[b][:seq[b]], ix_keys[b][:seq[b]]
        ref = R.step(page, mp, n_pages, n_tok, new, list(map(int, seq)), list(map(int, held)), table, free, count)
        coli.colibri_kv_step(d, B, n_tok, ints(torch, new), t["seq"], t["held"], t["table"], t["free"], t["count"], t["seq"],
                             t["held"], t["count"], t["q_start"], t["position"], t["slot"], t["status"], st)
        lat = torch.randn((n_tok, W), device="cuda").to(torch.bfloat16)
        coli.colibri_kv_append(d, n_tok, t["q_start"][B:], lat, W, lat[:, V:], W, t["slot"], cache, st)
        q = (torch.randn((n_tok, heads, W), device="cuda") * 1.5).to(torch.bfloat16)
        table, free, count = ref["table"], ref["free"], ref["count_out"]
        seq, held, qs = ref["seq_out"].astype(int), ref["held_out"].astype(int), ref["q_start"]
        N = int(qs[-1])
        sel = torch.full((n_tok, topk), -1, dtype=torch.int32, device="cuda")
        for b in range(B):
            if new[b] <= 0:
                if new[b] < 0:
                    keys_all[b], ix_keys[b] = np.zeros((0, W)), ix_keys[b][:0]
                continue
            keys_all[b] = np.concatenate([keys_all[b], lat[qs[b]:qs[b + 1]].double().cpu().numpy()])
            ix_keys[b] = torch.cat([ix_keys[b], torch.randn((new[b], 128), device="cuda").to(torch.bfloat16)]).contiguous()
            qi = torch.randn((new[b], 64, 128), device="cuda").to(torch.bfloat16)
            wi = torch.rand((new[b], 64), device="cuda")
            coli.colibri_indexer_topk(new[b], len(ix_keys[b]), int(seq[b]) - new[b], 64, 128, topk, qi, wi, ix_keys[b],
                                      sel[qs[b]:], ix_ws, ix_ws.numel(), st)
        out = torch.zeros((n_tok, heads, V), dtype=torch.bfloat16, device="cuda")
        coli.colibri_kv_attention(d, B, n_tok, heads, W ** -0.5, q, heads * W, W, cache, t["table"], t["q_start"], t["seq"],
                                  sel, topk, out, None, ws, n_ws, st)
        x = (out[:N].float().reshape(N, -1) @ up).to(torch.bfloat16)
        y = dl.forward(x.contiguous())
        torch.cuda.synchronize()
        assert int(t["status"][0]) == 0 and coli.colibri_kv_check_status(ws, st) == 0 and dl.plan.check_status(dl.ws) == 0
        np.testing.assert_array_equal(t["table"].cpu().numpy(), table)
        np.testing.assert_array_equal(t["q_start"].cpu().numpy(), qs)
        np.testing.assert_array_equal(t["slot"].cpu().numpy()[:N], ref["slot"])
        flat = cache.double().cpu().numpy().ravel()
        view = R.Cache(flat, page, page * W)
        for b in range(B):
            for j in range(len(keys_all[b])):
                np.testing.assert_array_equal(view.row(table[b][j // page], j % page), keys_all[b][j])
        o, _, tol, _, done = R.attention(q[:N].double().cpu().numpy(), view, table, qs, list(seq), W ** -0.5, 2.0 ** -7,
                                         sel=sel[:N].cpu().numpy())
        assert done.all()
        assert (np.abs(out[:N].double().cpu().numpy() - o) <= tol).all()
        assert torch.isfinite(y).all() and (out[N:] == 0).all()
        back = [1, 2, 0]
        back = [min(back[b], max(new[b] - 1, 0)) for b in range(B)]
    dl.close()
