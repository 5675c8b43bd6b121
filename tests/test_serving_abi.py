"""Refusals of the serving entry points (routing, paged cache, attention): argument checks before any CUDA call (no GPU)."""
import ctypes

import pytest

import quantized_expert_ffn_bias_gb300 as coli

P = 1 << 20          # an aligned address that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def built():
    coli.build()


def refused(status, fn, *a):
    with pytest.raises(coli.ColiError) as e:
        fn(*a)
    assert e.value.status == status
    assert len(str(e.value)) > 25


ROUTE = dict(E=256, k=8, score=0, n_group=8, topk_group=4, group_score=0, renorm=1, scale=1.0)


@pytest.mark.parametrize("bad,status", [
    (dict(E=0), coli.COLI_EINVAL), (dict(k=0), coli.COLI_EINVAL), (dict(E=2048), coli.COLI_EUNSUPPORTED),
    (dict(score=2), coli.COLI_EINVAL), (dict(score=-1), coli.COLI_EINVAL), (dict(n_group=7), coli.COLI_EINVAL),
    (dict(n_group=0), coli.COLI_EINVAL), (dict(n_group=64, topk_group=1, k=1), coli.COLI_EINVAL),
    (dict(topk_group=0), coli.COLI_EINVAL), (dict(topk_group=9), coli.COLI_EINVAL), (dict(group_score=2), coli.COLI_EINVAL),
    (dict(k=33), coli.COLI_EINVAL), (dict(E=16, n_group=8, topk_group=2, k=5), coli.COLI_EINVAL),
    (dict(E=8, n_group=8, topk_group=2, k=2), coli.COLI_EINVAL),          # top-2 of groups of one
    (dict(renorm=2), coli.COLI_EINVAL), (dict(scale=float("nan")), coli.COLI_EINVAL),
])
def test_route_description(bad, status):
    d = coli.coli_route_desc(**{**ROUTE, **bad})
    refused(status, coli.colibri_moe_route, d, 1, P, 1, max(d.E, 1), None, P, P, None)


def test_route_arguments():
    d = coli.coli_route_desc(**ROUTE)
    go = coli.colibri_moe_route
    refused(coli.COLI_EINVAL, go, d, -1, P, 1, 256, None, P, P, None)
    refused(coli.COLI_EUNSUPPORTED, go, d, 1, P, 3, 256, None, P, P, None)
    refused(coli.COLI_EINVAL, go, d, 1, P, 1, 255, None, P, P, None)
    refused(coli.COLI_EINVAL, go, d, 1, None, 1, 256, None, P, P, None)
    refused(coli.COLI_EINVAL, go, d, 1, P, 1, 256, None, None, P, None)
    refused(coli.COLI_EINVAL, go, d, 1, P, 1, 256, None, P, None, None)
    refused(coli.COLI_EALIGN, go, d, 1, P + 2, 1, 256, None, P, P, None)
    refused(coli.COLI_EALIGN, go, d, 1, P + 1, 0, 256, None, P, P, None)
    refused(coli.COLI_EALIGN, go, d, 1, P, 1, 256, P + 2, P, P, None)
    go(d, 0, None, 1, 256, None, None, None, None)                        # no tokens: nothing to do
    assert coli.lib().colibri_moe_route(None, 1, P, 1, 256, None, P, P, None) == coli.COLI_EINVAL


def test_set_route_checks_against_the_plan():
    p = coli.Plan(T_max=4, d=512, d_ff=256, E=256, k=8, routed_scale=2.5, qtype=coli.COLI_Q_INT4_G128, xtype=coli.COLI_X_BF16)
    p.set_route(coli.coli_route_desc(**ROUTE))
    p.set_route(None)
    refused(coli.COLI_EINVAL, p.set_route, coli.coli_route_desc(**{**ROUTE, "E": 128}))
    refused(coli.COLI_EINVAL, p.set_route, coli.coli_route_desc(**{**ROUTE, "k": 4}))
    refused(coli.COLI_EINVAL, p.set_route, coli.coli_route_desc(**{**ROUTE, "renorm": 5}))
    assert coli.lib().colibri_moe_set_route(None, None) == coli.COLI_EINVAL
    p.close()


KV = dict(page_size=64, max_pages=10, n_pages=100, dtype=0, page_stride=64 * 576)


def kv(**kw):
    return coli.coli_kv_desc(**{**KV, **kw})


def step(d, B=2, n=4, **kw):
    names = ["new_len", "seq_len", "held", "block_table", "free_pages", "free_count", "seq_len_out", "held_out",
             "free_count_out", "q_start", "position", "slot", "status"]
    coli.colibri_kv_step(d, B, n, *[kw.get(x, P) for x in names], None)


def append(d, n=2, n_valid=None, latent=P, ls=512, rope=P, rs=64, slot=P, cache=P):
    coli.colibri_kv_append(d, n, n_valid, latent, ls, rope, rs, slot, cache, None)


def attn(d, B=1, n=2, H=64, scale=0.1, q=P, ts=64 * 576, hs=576, cache=P, table=P, q_start=P, seq=P, sel=None, topk=0, out=P,
         lse=None, ws=P, nbytes=1 << 40):
    coli.colibri_kv_attention(d, B, n, H, scale, q, ts, hs, cache, table, q_start, seq, sel, topk, out, lse, ws, nbytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(page_size=0), coli.COLI_EINVAL), (dict(max_pages=0), coli.COLI_EINVAL), (dict(n_pages=0), coli.COLI_EINVAL),
    (dict(page_stride=63 * 576), coli.COLI_EINVAL), (dict(page_stride=64 * 576 + 8), coli.COLI_EINVAL),
    (dict(n_pages=1 << 26), coli.COLI_EUNSUPPORTED), (dict(max_pages=1 << 26), coli.COLI_EUNSUPPORTED),
])
def test_cache_description(bad, status):
    for fn in (step, append, attn):
        refused(status, fn, kv(**bad))


def test_step_arguments():
    refused(coli.COLI_EINVAL, step, kv(), 0)
    refused(coli.COLI_EUNSUPPORTED, step, kv(), 8193)
    refused(coli.COLI_EINVAL, step, kv(), 2, -1)
    for name in ("new_len", "seq_len", "held", "block_table", "free_pages", "free_count", "seq_len_out", "held_out",
                 "free_count_out", "q_start", "position", "slot", "status"):
        with pytest.raises(coli.ColiError) as e:
            step(kv(), **{name: None})
        assert e.value.status == coli.COLI_EINVAL, name
        with pytest.raises(coli.ColiError) as e:
            step(kv(), **{name: P + 2})
        assert e.value.status == coli.COLI_EALIGN, name


def test_append_arguments():
    refused(coli.COLI_EINVAL, append, kv(), -1)
    append(kv(), 0, latent=None, rope=None, slot=None, cache=None)
    for bad in (dict(latent=None), dict(rope=None), dict(slot=None), dict(cache=None), dict(ls=-8), dict(rs=-8)):
        with pytest.raises(coli.ColiError) as e:
            append(kv(), **bad)
        assert e.value.status == coli.COLI_EINVAL
    for bad in (dict(latent=P + 8), dict(rope=P + 2), dict(cache=P + 8), dict(ls=516), dict(rs=68), dict(slot=P + 1),
                dict(n_valid=P + 2)):
        with pytest.raises(coli.ColiError) as e:
            append(kv(), **bad)
        assert e.value.status == coli.COLI_EALIGN


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), coli.COLI_EINVAL), (dict(n=-1), coli.COLI_EINVAL), (dict(H=0), coli.COLI_EINVAL),
    (dict(B=8193), coli.COLI_EUNSUPPORTED), (dict(H=1025), coli.COLI_EUNSUPPORTED),
    (dict(scale=float("nan")), coli.COLI_EINVAL), (dict(scale=float("inf")), coli.COLI_EINVAL),
    (dict(sel=P, topk=0), coli.COLI_EINVAL), (dict(sel=P, topk=(1 << 30) + 1), coli.COLI_EUNSUPPORTED), (dict(n=1 << 26), coli.COLI_EUNSUPPORTED),
    (dict(q=None), coli.COLI_EINVAL), (dict(cache=None), coli.COLI_EINVAL), (dict(table=None), coli.COLI_EINVAL),
    (dict(q_start=None), coli.COLI_EINVAL), (dict(seq=None), coli.COLI_EINVAL), (dict(out=None), coli.COLI_EINVAL),
    (dict(ws=None), coli.COLI_EINVAL), (dict(q=P + 8), coli.COLI_EALIGN), (dict(cache=P + 2), coli.COLI_EALIGN),
    (dict(out=P + 4), coli.COLI_EALIGN), (dict(ws=P + 128), coli.COLI_EALIGN), (dict(lse=P + 2), coli.COLI_EALIGN),
    (dict(sel=P + 2, topk=4), coli.COLI_EALIGN), (dict(ts=0), coli.COLI_EINVAL), (dict(hs=-576), coli.COLI_EINVAL),
    (dict(ts=64 * 576 + 4), coli.COLI_EALIGN), (dict(hs=580), coli.COLI_EALIGN), (dict(nbytes=1000), coli.COLI_EWORKSPACE),
])
def test_attention_arguments(bad, status):
    refused(status, lambda: attn(kv(), **bad))


def test_attention_other_refusals():
    refused(coli.COLI_EUNSUPPORTED, attn, kv(dtype=coli.COLI_X_F32))
    refused(coli.COLI_EUNSUPPORTED, attn, kv(dtype=7))
    attn(kv(), n=0, q=None, cache=None, table=None, q_start=None, seq=None, out=None, ws=None)
    refused(coli.COLI_EINVAL, coli.colibri_kv_attention_workspace_size, 0, 1, 1)
    refused(coli.COLI_EINVAL, coli.colibri_kv_attention_workspace_size, 1, -1, 1)
    refused(coli.COLI_EUNSUPPORTED, coli.colibri_kv_attention_workspace_size, 1, 1 << 26, 64)
    n = [coli.colibri_kv_attention_workspace_size(4, t, 64) for t in (1, 1000, 100000)]
    assert n[0] <= n[1] < n[2]
    v = ctypes.c_int32()
    assert coli.lib().colibri_kv_check_status(None, ctypes.byref(v), None) == coli.COLI_EINVAL
