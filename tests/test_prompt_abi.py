"""Rotary frequencies, and refusals of the prompt operators' entry points: argument checks before any CUDA call (no GPU)."""
import ctypes
import math

import pytest

import quantized_expert_ffn_bias_gb300 as coli

P = 1 << 20          # an aligned address that no refused call reads
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    coli.build()


def refused(code, fn, *a, **kw):
    with pytest.raises(coli.ColiError) as e:
        fn(*a, **kw)
    assert e.value.status == code
    assert len(str(e.value)) > 25


def rope(**kw):
    d = dict(dim=64, layout=0, scaling=3, amplitude=1.0, base=10000.0, factor=40.0, original_len=4096.0, beta_fast=32.0, beta_slow=1.0)
    return coli.coli_rope_desc(**{**d, **kw})


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("dim,base,original", [(64, 10000.0, 4096.0), (2, 10000.0, 4096.0), (256, 5e5, 8192.0), (40, 1e6, 32768.0), (64, 1.5, 100.0),
                                              (128, 10000.0, 4.0)])
def test_frequencies(scaling, dim, base, original):
    torch = pytest.importorskip("torch")
    assert torch is not None
    from tests import prompt_ref as R
    f = coli.colibri_rope_frequencies(rope(dim=dim, base=base, factor=8.0, original_len=original,
                                           scaling={"none": 0, "linear": 1, "ntk": 2, "yarn": 3}[scaling]))
    want = R.frequencies(dim, scaling, base=base, factor=8.0, original=original)
    assert len(f) == dim // 2
    for got, w in zip(f, want):
        # powers in 64 bits (a few 2^-52, times the exponent's size) and half a unit of the table
        assert abs(got - w / (2 * math.pi) * 2.0 ** 64) <= 1 + got * 2.0 ** -44
        assert 0 <= got < 2 ** 62


@pytest.mark.parametrize("bad", [
    dict(dim=0), dict(dim=63), dict(dim=258), dict(dim=-2), dict(layout=2), dict(layout=-1), dict(scaling=4), dict(scaling=-1), dict(amplitude=NAN),
    dict(amplitude=INF), dict(base=1.0), dict(base=NAN), dict(base=INF), dict(base=-5.0), dict(factor=0.5), dict(factor=NAN), dict(factor=INF),
    dict(original_len=0.0), dict(original_len=NAN), dict(original_len=INF), dict(beta_slow=0.0), dict(beta_slow=32.0), dict(beta_fast=NAN),
    dict(beta_fast=INF)])
def test_frequencies_refuse(bad):
    refused(coli.COLI_EINVAL, coli.colibri_rope_frequencies, rope(**bad))


def test_frequencies_null():
    f = (ctypes.c_uint64 * 32)()
    assert coli.lib().colibri_rope_frequencies(None, f) == coli.COLI_EINVAL
    assert coli.lib().colibri_rope_frequencies(ctypes.byref(rope()), None) == coli.COLI_EINVAL
    assert coli.lib().colibri_rope(None, 0, 1, None, 1, P, P, P, 64, 64, P, 64, 64, None) == coli.COLI_EINVAL


def turn(d=None, dtype=0, n=2, n_valid=None, H=4, pos=P, freq=P, x=P, xt=256, xh=64, out=P, ot=256, oh=64):
    coli.colibri_rope(d or rope(), dtype, n, n_valid, H, pos, freq, x, xt, xh, out, ot, oh, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=rope(dim=3)), coli.COLI_EINVAL), (dict(d=rope(layout=7)), coli.COLI_EINVAL), (dict(d=rope(amplitude=INF)), coli.COLI_EINVAL),
    (dict(n=-1), coli.COLI_EINVAL), (dict(H=0), coli.COLI_EINVAL), (dict(H=1025), coli.COLI_EUNSUPPORTED), (dict(dtype=3), coli.COLI_EUNSUPPORTED),
    (dict(dtype=-1), coli.COLI_EUNSUPPORTED), (dict(pos=None), coli.COLI_EINVAL), (dict(freq=None), coli.COLI_EINVAL), (dict(x=None), coli.COLI_EINVAL),
    (dict(out=None), coli.COLI_EINVAL), (dict(pos=P + 2), coli.COLI_EALIGN), (dict(freq=P + 4), coli.COLI_EALIGN), (dict(x=P + 1), coli.COLI_EALIGN),
    (dict(out=P + 1), coli.COLI_EALIGN), (dict(dtype=1, x=P + 2), coli.COLI_EALIGN), (dict(n_valid=P + 1), coli.COLI_EALIGN),
    (dict(xt=-1), coli.COLI_EINVAL), (dict(xh=-64), coli.COLI_EINVAL), (dict(ot=0), coli.COLI_EINVAL), (dict(ot=-5), coli.COLI_EINVAL),
    (dict(oh=63), coli.COLI_EINVAL)])
def test_rope_refuses(kw, status):
    refused(status, turn, **kw)


@pytest.mark.parametrize("kw", [dict(ot=63), dict(ot=1, oh=512), dict(H=1, ot=40), dict(n=1, oh=32), dict(xt=512), dict(xh=128), dict(ot=320),
                                dict(H=1, ot=64), dict(xt=0, x=P, out=P)])
def test_rope_refuses_outputs_that_overlap(kw):
    """Rows or heads nearer than dim, and rotation in place with other strides."""
    refused(coli.COLI_EINVAL, turn, **kw)


def test_rope_of_nothing():
    turn(n=0, pos=None, freq=None, x=None, out=None)


KV = dict(page_size=64, max_pages=10, n_pages=100, dtype=0, page_stride=64 * 576)


def kv(**kw):
    return coli.coli_kv_desc(**{**KV, **kw})


def append(d=None, r=None, n=2, n_valid=None, latent=P, ls=512, gain=P, eps=1e-6, rot=P, rs=64, pos=P, freq=P, slot=P, cache=P):
    coli.colibri_kv_append_rope(d or kv(), r or rope(), n, n_valid, latent, ls, gain, eps, rot, rs, pos, freq, slot, cache, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=kv(page_size=0)), coli.COLI_EINVAL), (dict(d=kv(dtype=1)), coli.COLI_EUNSUPPORTED), (dict(r=rope(dim=62)), coli.COLI_EINVAL),
    (dict(r=rope(dim=65)), coli.COLI_EINVAL), (dict(r=rope(layout=3)), coli.COLI_EINVAL), (dict(r=rope(amplitude=NAN)), coli.COLI_EINVAL),
    (dict(n=-1), coli.COLI_EINVAL), (dict(eps=-1e-6), coli.COLI_EINVAL), (dict(eps=NAN), coli.COLI_EINVAL), (dict(eps=INF), coli.COLI_EINVAL),
    (dict(latent=None), coli.COLI_EINVAL), (dict(rot=None), coli.COLI_EINVAL), (dict(slot=None), coli.COLI_EINVAL), (dict(cache=None), coli.COLI_EINVAL),
    (dict(pos=None), coli.COLI_EINVAL), (dict(freq=None), coli.COLI_EINVAL), (dict(ls=-8), coli.COLI_EINVAL), (dict(rs=-8), coli.COLI_EINVAL),
    (dict(latent=P + 8), coli.COLI_EALIGN), (dict(rot=P + 2), coli.COLI_EALIGN), (dict(gain=P + 4), coli.COLI_EALIGN), (dict(cache=P + 8), coli.COLI_EALIGN),
    (dict(ls=516), coli.COLI_EALIGN), (dict(rs=68), coli.COLI_EALIGN), (dict(slot=P + 1), coli.COLI_EALIGN), (dict(n_valid=P + 2), coli.COLI_EALIGN),
    (dict(pos=P + 1), coli.COLI_EALIGN), (dict(freq=P + 4), coli.COLI_EALIGN)])
def test_append_rope_refuses(kw, status):
    refused(status, append, **kw)


def test_append_rope_of_nothing():
    append(n=0, latent=None, gain=None, rot=None, pos=None, freq=None, slot=None, cache=None)
    append(n=0, gain=None, eps=NAN)                    # not read without a gain
    assert coli.lib().colibri_kv_append_rope(ctypes.byref(kv()), None, 1, None, P, 512, None, 0.0, P, 64, P, P, P, P, None) == coli.COLI_EINVAL
    assert coli.lib().colibri_kv_append_rope(None, ctypes.byref(rope()), 1, None, P, 512, None, 0.0, P, 64, P, P, P, P, None) == coli.COLI_EINVAL


def gather(d=None, B=2, n=100, seq=P, table=P, cache=P, start=P, latent=P, ls=512, rot=P, rs=64, status=P):
    coli.colibri_kv_gather(d or kv(), B, n, seq, table, cache, start, latent, ls, rot, rs, status, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=kv(max_pages=0)), coli.COLI_EINVAL), (dict(B=0), coli.COLI_EINVAL), (dict(B=8193), coli.COLI_EUNSUPPORTED), (dict(n=-1), coli.COLI_EINVAL),
    (dict(n=2**31 - 1), coli.COLI_EUNSUPPORTED), (dict(seq=None), coli.COLI_EINVAL), (dict(table=None), coli.COLI_EINVAL), (dict(cache=None), coli.COLI_EINVAL),
    (dict(start=None), coli.COLI_EINVAL), (dict(latent=None), coli.COLI_EINVAL), (dict(rot=None), coli.COLI_EINVAL), (dict(status=None), coli.COLI_EINVAL),
    (dict(seq=P + 1), coli.COLI_EALIGN), (dict(start=P + 2), coli.COLI_EALIGN), (dict(status=P + 2), coli.COLI_EALIGN), (dict(cache=P + 8), coli.COLI_EALIGN),
    (dict(latent=P + 8), coli.COLI_EALIGN), (dict(rot=P + 8), coli.COLI_EALIGN), (dict(ls=504), coli.COLI_EINVAL), (dict(rs=56), coli.COLI_EINVAL),
    (dict(ls=516), coli.COLI_EALIGN), (dict(rs=68), coli.COLI_EALIGN)])
def test_gather_refuses(kw, status):
    refused(status, gather, **kw)


def attend(dtype=0, B=2, n=4, m=8, H=4, scale=0.1, q=P, qt=768, qh=192, k=P, kt=1024, kh=256, r=P, rs=64, v=P, vt=1024, vh=256, qs=P, ks=P, out=P,
           lse=None, ws=P, nbytes=1 << 40):
    coli.colibri_prompt_attention(dtype, B, n, m, H, scale, q, qt, qh, k, kt, kh, r, rs, v, vt, vh, qs, ks, out, lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), coli.COLI_EUNSUPPORTED), (dict(dtype=9), coli.COLI_EUNSUPPORTED), (dict(B=0), coli.COLI_EINVAL), (dict(B=8193), coli.COLI_EUNSUPPORTED),
    (dict(n=-1), coli.COLI_EINVAL), (dict(m=-1), coli.COLI_EINVAL), (dict(H=0), coli.COLI_EINVAL), (dict(H=1025), coli.COLI_EUNSUPPORTED),
    (dict(n=2**31 - 1), coli.COLI_EUNSUPPORTED), (dict(m=2**31 - 1), coli.COLI_EUNSUPPORTED), (dict(scale=NAN), coli.COLI_EINVAL),
    (dict(scale=3e38), coli.COLI_EINVAL), (dict(q=None), coli.COLI_EINVAL), (dict(k=None), coli.COLI_EINVAL), (dict(r=None), coli.COLI_EINVAL),
    (dict(v=None), coli.COLI_EINVAL), (dict(qs=None), coli.COLI_EINVAL), (dict(ks=None), coli.COLI_EINVAL), (dict(out=None), coli.COLI_EINVAL),
    (dict(ws=None), coli.COLI_EINVAL), (dict(q=P + 8), coli.COLI_EALIGN), (dict(k=P + 2), coli.COLI_EALIGN), (dict(r=P + 8), coli.COLI_EALIGN),
    (dict(v=P + 4), coli.COLI_EALIGN), (dict(out=P + 8), coli.COLI_EALIGN), (dict(ws=P + 128), coli.COLI_EALIGN), (dict(lse=P + 2), coli.COLI_EALIGN),
    (dict(qs=P + 2), coli.COLI_EALIGN), (dict(ks=P + 1), coli.COLI_EALIGN), (dict(qt=0), coli.COLI_EINVAL), (dict(qh=-192), coli.COLI_EINVAL),
    (dict(kt=-1024), coli.COLI_EINVAL), (dict(kh=0), coli.COLI_EINVAL), (dict(rs=0), coli.COLI_EINVAL), (dict(vt=0), coli.COLI_EINVAL),
    (dict(vh=0), coli.COLI_EINVAL), (dict(qt=772), coli.COLI_EALIGN), (dict(kh=257), coli.COLI_EALIGN), (dict(rs=66), coli.COLI_EALIGN),
    (dict(vt=1 << 38), coli.COLI_EUNSUPPORTED), (dict(nbytes=1000), coli.COLI_EWORKSPACE)])
def test_prompt_attention_refuses(kw, status):
    refused(status, attend, **kw)


def test_prompt_attention_of_nothing():
    attend(n=0, q=None, k=None, r=None, v=None, qs=None, ks=None, out=None, ws=None)
    assert coli.colibri_prompt_attention_workspace_size(1, 0, 0, 1) % 256 == 0
    refused(coli.COLI_EINVAL, coli.colibri_prompt_attention_workspace_size, 0, 1, 1, 1)
    refused(coli.COLI_EINVAL, coli.colibri_prompt_attention_workspace_size, 1, 1, -1, 1)
