"""Attention over the paged cache where its arithmetic or its arguments are at an edge (needs a GB300): very low and very
uneven scores, row offsets that do not ascend or pass the batch, lengths of the step's token rows at the type's limit, and
a pipeline wait that runs out."""
from __future__ import annotations

import numpy as np
import pytest

from tests import serving_ref as R
from tests.test_gpu_kv import Batch, V, W, ints, selected, torch_cuda  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def rows_of(b, request):
    """The cached rows of a request's keys, in key order: a view to read, and a function that writes them."""
    n = b.lens[request]
    pages = np.asarray(b.table[request])[np.arange(n) // b.page]
    at = pages.astype(np.int64) * (b.stride // W) + np.arange(n) % b.page
    flat = b.cache.view(-1, W)
    idx = b.torch.from_numpy(at).cuda()
    return flat, idx


def shift_scores(b, request, nats):
    """Lower (or raise) the scores of a request's keys by about nats[j], the same for every head: the last rotary value of
    the queries is 48, so that the keys' last value v adds 48 v / 24 to a score."""
    flat, idx = rows_of(b, request)
    b.q[..., W - 1] = 48.0
    add = b.torch.as_tensor(np.broadcast_to(np.asarray(nats, np.float32) / 2.0, (b.lens[request],)).copy()).cuda()
    flat[idx, W - 1] = add.to(b.dt)


FORMS = [(64, "bf16"), (64, "f16"), (16, "bf16"), (16, "f16")]      # TMA boxes, copied rows


@pytest.mark.parametrize("page,dtype", FORMS)
@pytest.mark.parametrize("nats", [-95.0, -150.0, -1000.0])
def test_attention_every_score_very_low(torch_cuda, page, dtype, nats):
    """One key, 300 keys and a chunk whose scores all lie far below the smallest power of two of fp32."""
    for lens, new in (([1], [1]), ([300], [2]), ([150, 1], [150, 1])):
        b = Batch(torch_cuda, lens, new, 16, page, dtype=dtype, seed=80)
        for i in range(len(lens)):
            shift_scores(b, i, nats)
        out, z = b.check()
        assert torch_cuda.isfinite(out).all() and torch_cuda.isfinite(z).all()


@pytest.mark.parametrize("page,dtype", FORMS)
@pytest.mark.parametrize("nats", [-100.0, -1000.0])
def test_attention_first_tile_very_low(torch_cuda, page, dtype, nats):
    """Very low scores in the first tile, or in all tiles but the last, and higher ones behind; the reverse order."""
    for low in (slice(0, 128), slice(0, 500), slice(100, 700)):
        shift = np.zeros(700)
        shift[low] = nats
        b = Batch(torch_cuda, [700, 700], [2, 1], 16, page, dtype=dtype, seed=81)
        shift_scores(b, 0, shift)
        shift_scores(b, 1, shift)
        out, z = b.check()
        assert torch_cuda.isfinite(out).all() and torch_cuda.isfinite(z).all()


@pytest.mark.parametrize("page,dtype", FORMS)
def test_attention_cut_runs_of_very_low_scores(torch_cuda, page, dtype):
    """A request cut over the card: runs that see very low scores alone, next to runs that do not; and all of them low."""
    for shift in (np.where(np.arange(12000) < 8000, -200.0, 0.0), np.where(np.arange(12000) < 5000, 0.0, -2000.0),
                  np.full(12000, -300.0)):
        b = Batch(torch_cuda, [12000], [1], 16, page, dtype=dtype, seed=82)
        shift_scores(b, 0, shift)
        out, z = b.check()
        assert torch_cuda.isfinite(out).all() and torch_cuda.isfinite(z).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("empty", [0, 128, 300])
def test_attention_selected_keys_of_very_low_scores(torch_cuda, dtype, empty):
    """Selections whose first tiles hold no entry and whose keys all score very low."""
    lens, new = [900, 700], [2, 1]
    b = Batch(torch_cuda, lens, new, 64, 64, dtype=dtype, seed=83)
    shift_scores(b, 0, -120.0)
    shift_scores(b, 1, -900.0)
    sel = selected(np.random.default_rng(83), lens, new, 600)
    sel[:, :empty] = -1
    out, z = b.check(sel=sel)
    assert torch_cuda.isfinite(out).all() and torch_cuda.isfinite(z).all()


@pytest.mark.parametrize("starts", [[0, 5, 4], [3, 0, 4], [0, 9, 2], [9, 8, 4], [0, 2, -1], [0, -5, 4]])
@pytest.mark.parametrize("page", [64, 16])
def test_attention_refuses_any_q_start_that_descends(torch_cuda, starts, page):
    """Also where the entries lie outside the batch: nothing is written, the status says so."""
    b = Batch(torch_cuda, [300, 100], [2, 2], 64, page, seed=85)
    b.q_start = np.array(starts, np.int32)
    out, z = b.run(status=R.TOKENS)
    assert (out == 3.0).all() and (z == 3.0).all()


@pytest.mark.parametrize("page", [64, 16])
def test_attention_rows_of_a_request_that_passes_the_batch(torch_cuda, page):
    """A request of five new tokens of which the batch holds two: those are its first two, at their own positions."""
    b = Batch(torch_cuda, [300, 100], [2, 5], 64, page, seed=86)
    cache = R.Cache(b.cache.double().cpu().numpy().ravel(), b.page, b.stride)
    ref, lse, tol, tol_lse, _ = R.attention(b.q.double().cpu().numpy(), cache, b.table, b.q_start, b.lens, b.scale,
                                            torch_cuda.finfo(b.dt).eps)
    b.q, b.N = b.q[:4].contiguous(), 4
    out, z = b.run()
    assert (np.abs(out.double().cpu().numpy() - ref[:4]) <= tol[:4]).all()
    assert (np.abs(z.double().cpu().numpy() - lse[:4]) <= tol_lse[:4]).all()


@pytest.mark.parametrize("n_tokens", [(1 << 31) - 1, (1 << 31) - 2])
def test_step_of_as_many_rows_as_the_type_counts(torch_cuda, n_tokens):
    """Room for 2^31 - 1 token rows: the sums of new tokens do not wrap.  Only the rows before q_start[B] are written, so
    the arrays here hold no more than those."""
    torch = torch_cuda
    import quantized_expert_ffn_bias_gb300 as coli
    page, mp, n_pages = 16, 4, 12
    new, seq, held = [3, 0, 20, -1, 1], [5, 0, 0, 7, 16], [1, 0, 0, 1, 1]
    table = np.full((5, mp), -1, np.int32)
    table[0, 0], table[3, 0], table[4, 0] = 4, 5, 6
    free = np.array([0, 1, 2, 3, 7, 8, 9, 10, 11, -1, -1, -1], np.int32)
    want = R.step(page, mp, n_pages, n_tokens, new, seq, held, table, free, 9)
    t = {k: ints(torch, v) for k, v in dict(new=new, seq=seq, held=held, table=table, free=free, count=[9], seq_out=[0] * 5,
                                            held_out=[0] * 5, count_out=[0], q_start=[0] * 6, position=[-9] * 64,
                                            slot=[-9] * 64, status=[0]).items()}
    d = coli.coli_kv_desc(page, mp, n_pages, 0, page * W)
    coli.colibri_kv_step(d, 5, n_tokens, *t.values(), torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in t.items()}
    for k in ("seq_out", "held_out", "q_start", "table", "free"):
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    n = len(want["position"])
    np.testing.assert_array_equal(got["position"][:n], want["position"])
    np.testing.assert_array_equal(got["slot"][:n], want["slot"])
    assert (got["position"][n:] == -9).all() and got["status"][0] == want["status"] == 0
    assert got["count_out"][0] == want["count_out"]


def test_attention_scores_below_any_reference(torch_cuda):
    """Finite scores of -5e34, equal for all keys (so the result is the mean of their values), in a unit cut over CTAs of
    which half see no key.  Weights are 1, their sum and the products' sums in fp32: 2^-23 a term, then one rounding."""
    torch = torch_cuda
    b = Batch(torch, [5000], [1], 64, 64, seed=87)
    flat, idx = rows_of(b, 0)
    b.q[..., W - 1] = 2.0 ** 60
    flat[idx, W - 1] = -2.0 ** 60
    sel = selected(np.random.default_rng(87), [5000], [1], 2048)
    sel[0, :1024] = -1
    out, z = b.run(sel=sel)
    v = flat[idx[torch.from_numpy(sel[0, 1024:]).cuda().long()], :V].double()
    want, mag = v.mean(0), v.abs().mean(0)
    tol = 2.0 ** -23 * 1100 * mag + torch.finfo(b.dt).eps / 2 * want.abs() * 1.01
    assert ((out[0].double() - want).abs() <= tol).all()
    s = -(2.0 ** 120) * b.scale
    assert ((z.double() - s).abs() <= 2.0 ** -21 * abs(s)).all()


@pytest.mark.parametrize("page", [64, 16])
def test_attention_many_small_weights_in_fp16(torch_cuda, page):
    """One strong key, then 20,000 whose weights are 2^-25 of it: together 2^-10.7 of the weights, times values of 1,000,
    which the weights' rounding to fp16 must not lose.  The largest weight is kept above 2^6, so what a weight loses below
    fp16's normal range is half of 2^-24 of 2^6 at most: the bound's `tiny` is 2^-7 of the one for a largest weight of 1/2.
    As many requests as there are SMs share the keys, so that no request is cut (a part without the strong key would have
    a reference of its own)."""
    torch = torch_cuda
    n, B = 20001, torch.cuda.get_device_properties(0).multi_processor_count
    b = Batch(torch, [n], [1], 2, page, dtype="f16", seed=88)
    b.scale = float(np.log(2.0))                       # scores in log2 units are the products themselves
    b.q.zero_()
    b.q[..., W - 1] = 1.0
    flat, idx = rows_of(b, 0)
    rows = torch.zeros((n, W), dtype=b.dt, device="cuda")
    rows[:, :V] = 1000.0
    rows[:, W - 1] = -25.015625
    rows[0, :V] = 0.0
    rows[0, W - 1] = 0.0
    flat[idx] = rows
    cache = R.Cache(b.cache.double().cpu().numpy().ravel(), b.page, b.stride)
    info = torch.finfo(b.dt)
    ref, lse, tol, tol_lse, _ = R.attention(b.q.double().cpu().numpy(), cache, b.table, b.q_start, b.lens, b.scale,
                                            info.eps, tiny=float(info.smallest_normal) * info.eps / 128)
    b.lens, b.table, b.q_start, b.N = [n] * B, np.repeat(b.table, B, 0), np.arange(B + 1, dtype=np.int32), B
    b.q = b.q.expand(B, -1, -1).contiguous()
    out, z = b.run()
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all(), (out[0, 0, :3], ref[0, 0, :3], tol[0, 0, :3])
    assert (np.abs(z.double().cpu().numpy() - lse) <= tol_lse).all()


def test_attention_fp16_references_rise_far(torch_cuda):
    """Scores that climb by 2 to 14 (log2) a tile, with fp16 weights up to 2^15: no weight or sum leaves its type."""
    torch = torch_cuda
    for step in (1.5, 5.0, 9.5):
        b = Batch(torch, [1300], [2], 16, 64, dtype="f16", seed=89)
        shift_scores(b, 0, np.arange(1300) // 128 * step)
        out, z = b.check()
        assert torch.isfinite(out).all() and torch.isfinite(z).all()


@pytest.mark.parametrize("lens,new,H,page,topk", [
    ([100], [1], 16, 64, 0), ([9000, 300], [3, 1], 64, 64, 0),        # TMA: one tile; tiles of a unit cut over the card
    ([100], [1], 16, 16, 0), ([9000, 300], [3, 1], 64, 16, 0),        # copied rows
    ([5000], [2], 64, 64, 512), ([60], [40], 64, 128, 0)])            # selected keys; several units
def test_attention_wait_that_runs_out(torch_cuda, lens, new, H, page, topk):
    """Copies that never come: the waits end after 2 ms, the status says so, the call and the next one on the same
    workspace return, and the next one is right."""
    import time
    torch = torch_cuda
    import quantized_expert_ffn_bias_gb300 as coli
    b = Batch(torch, lens, new, H, page, seed=90)
    sel = selected(np.random.default_rng(90), lens, new, topk) if topk else None
    want, lse = b.check(sel=sel)
    ws = torch.empty(coli.colibri_kv_attention_workspace_size(len(lens), b.N, H), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        coli.colibri_kv_debug_inject(coli.COLI_INJECT_WITHHOLD_STAGE, 2.0)
        try:
            t0 = time.perf_counter()
            b.run(sel=sel, ws=ws, status=coli.COLI_DEV_WAIT_TIMEOUT)
            assert time.perf_counter() - t0 < 0.5
        finally:
            coli.colibri_kv_debug_inject(0)
        out, z = b.run(sel=sel, ws=ws)
        assert torch.equal(out, want) and torch.equal(z, lse)
