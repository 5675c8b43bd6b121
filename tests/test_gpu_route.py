"""Routing from given logits on the GPU against the 64-bit form (needs a GB300): ids equal, weights within the fp32
arithmetic's error, and the layer forward with a routing set on its plan."""
from __future__ import annotations

import numpy as np
import pytest

import harness as H
import oracle as O
from tests import serving_ref as R
from tests.gpu_parity import check_output

pytestmark = pytest.mark.gpu

# expf 2 ulp, 1 + e, the quotient: 4 * 2^-23 a sigmoid.  Softmax: exp(z - m) 2 ulp and the rounding of its argument
# (2^-24 |z - m|, below 2^-24 * 40 where the weight matters), 1024 terms in sums of 32 and 5 levels (37 * 2^-24), the
# product with 1 / sum; then renormalising doubles it and adds three roundings.
W_TOL = 2 * (2 + 40 / 2 + 37 / 2 + 3) * 2.0 ** -23


@pytest.fixture(scope="module")
def torch_cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_expert_ffn_bias_gb300 as coli
    coli.build()
    return torch


def _desc(coli, E, k, score="sigmoid", groups=1, keep=1, gscore="top2", renorm=True, scale=2.5):
    return coli.coli_route_desc(E, k, {"sigmoid": 0, "softmax": 1}[score], groups, keep, {"top2": 0, "max": 1}[gscore],
                                int(renorm), scale)


def run_route(torch, z, bias, dtype="f32", pad=0, **kw):
    """z fp32 numpy [T][E] -> ids, weights, and the logits as the kernel read them (fp64)."""
    import quantized_expert_ffn_bias_gb300 as coli
    T, E = z.shape
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    buf = torch.full((T, E + pad), float("nan"), dtype=dt, device="cuda")
    buf[:, :E] = torch.from_numpy(z).cuda().to(dt)
    bd = torch.from_numpy(bias).cuda() if bias is not None else None
    k = kw["k"]
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    coli.colibri_moe_route(_desc(coli, E, **kw), T, buf, {"bf16": 0, "f32": 1, "f16": 2}[dtype], E + pad, bd, idx, w,
                           torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert (idx[T] == -7).all() and (w[T] == -7).all(), "rows behind the last token"
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy(), buf[:, :E].double().cpu().numpy()


def check(torch, z, bias, dtype="f32", pad=0, **kw):
    idx, w, zr = run_route(torch, z, bias, dtype, pad, **kw)
    ids, ws = R.route(zr, bias, **{"scale": 2.5, **kw})
    np.testing.assert_array_equal(idx, ids)
    np.testing.assert_allclose(w, ws, rtol=W_TOL, atol=2.5 * 1e-37)


CASES = [
    dict(T=1, E=256, k=8, groups=8, keep=4),
    dict(T=3, E=256, k=8, groups=8, keep=4, gscore="max", score="softmax", renorm=False),
    dict(T=130, E=160, k=6, groups=8, keep=3, gscore="max", score="softmax", renorm=False, bias=None),
    dict(T=65, E=384, k=8, groups=1, keep=1, dtype="bf16"),
    dict(T=65, E=64, k=6, score="softmax", dtype="f16", bias=None, pad=3),
    dict(T=33, E=1024, k=32, groups=32, keep=5, dtype="bf16", pad=1),
    dict(T=257, E=8, k=2, score="softmax", bias=None, dtype="bf16"),
    dict(T=7, E=1, k=1),
    dict(T=70, E=384, k=8, groups=8, keep=4),
    dict(T=70, E=320, k=8, groups=16, keep=4, dtype="bf16", bias=None),
    dict(T=40, E=512, k=16, groups=8, keep=3, dtype="f16"),
    dict(T=40, E=1000, k=8, groups=8, keep=3),
    dict(T=5, E=33, k=32, groups=3, keep=3),
    dict(T=5, E=62, k=4, groups=31, keep=2, renorm=False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{a}{b}" for a, b in c.items()))
def test_route_matches_64_bits(torch_cuda, case):
    c = dict(case)
    T, E, dtype, pad, has_bias = c.pop("T"), c["E"], c.pop("dtype", "f32"), c.pop("pad", 0), c.pop("bias", True)
    c.pop("E")
    rng = np.random.default_rng(T * 1000 + E)
    z = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if has_bias else None
    check(torch_cuda, z, bias, dtype, pad, **c)


def test_route_close_scores_are_told_apart(torch_cuda):
    """Logits a few fp32 steps apart, far into the sigmoid's flat part: fp32 scores tie or swap, the exact ones do not."""
    rng = np.random.default_rng(5)
    T, E = 64, 128
    base = rng.choice(np.array([-20.0, -3.0, 0.5, 9.0, 16.5], np.float32), (T, 1)) * np.ones((1, E), np.float32)
    z = base + (rng.integers(-40, 41, (T, E)) * np.spacing(np.abs(base))).astype(np.float32)
    for kw in (dict(score="sigmoid"), dict(score="softmax"), dict(score="sigmoid", groups=8, keep=3, gscore="max"),
               dict(score="softmax", groups=8, keep=3, gscore="max")):
        check(torch_cuda, z.astype(np.float32), None, k=9, **kw)
        check(torch_cuda, z.astype(np.float32), np.full(E, 0.25, np.float32), k=9, **kw)


def test_route_ties_take_the_lower_id(torch_cuda):
    for score in ("sigmoid", "softmax"):
        check(torch_cuda, np.zeros((4, 96), np.float32), None, k=5, score=score, groups=6, keep=3)
        rng = np.random.default_rng(9)
        z = rng.integers(-2, 3, (200, 256)).astype(np.float32)          # many equal logits
        check(torch_cuda, z, None, "bf16", k=8, score=score, groups=8, keep=4)


def test_route_special_values(torch_cuda):
    """Infinities, NaN and the type's lowest value among logits and biases; rows with nothing to choose from."""
    rng = np.random.default_rng(11)
    E = 64
    z = rng.standard_normal((8, E)).astype(np.float32)
    z[0, 10:] = -np.inf
    z[1] = -np.inf
    z[2, 5] = np.inf
    z[3, [4, 40]] = np.inf
    z[4, ::2] = np.nan
    z[5] = np.nan
    z[6, 1:] = np.finfo(np.float32).min
    z[7, :3] = np.finfo(np.float32).max
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
    shut = bias.copy()
    shut[8:16] = -np.inf
    shut[20] = np.nan
    low = bias.copy()
    low[:40] = np.finfo(np.float32).min
    for b in (None, bias, shut, low):
        for kw in (dict(score="sigmoid"), dict(score="softmax"), dict(score="softmax", renorm=False),
                   dict(score="sigmoid", groups=8, keep=2), dict(score="softmax", groups=8, keep=4, gscore="max")):
            check(torch_cuda, z, b, k=6, **kw)


@pytest.mark.parametrize("E,groups", [(64, 8), (62, 31), (96, 4), (160, 5), (384, 8), (1000, 8)])
def test_route_infinite_biases(torch_cuda, E, groups):
    """Biases that force experts in (+infinity) or shut them out (-infinity): fewer and more of them than there are
    picks, whole groups, groups that are not whole lanes; sums that pass fp32's largest value."""
    rng = np.random.default_rng(E)
    z = rng.standard_normal((16, E)).astype(np.float32)
    size, k = E // groups, 4
    base = (rng.standard_normal(E) * 0.05).astype(np.float32)
    biases = []
    for n in (1, 3, k, k + 3):
        b = base.copy()
        b[rng.choice(E, n, replace=False)] = np.inf
        biases.append(b.copy())
        b[rng.choice(E, E // 2, replace=False)] = -np.inf
        biases.append(b)
    shut = base.copy()
    shut[size - 1:-size] = -np.inf
    force = base.copy()
    force[size + 1:2 * size] = np.inf
    big = base.copy()
    big[size:] = np.finfo(np.float32).max
    biases += [shut, force, big, np.full(E, np.inf, np.float32), np.full(E, -np.inf, np.float32)]
    for b in biases:
        for kw in (dict(score="sigmoid"), dict(score="softmax"), dict(score="sigmoid", groups=groups, keep=2),
                   dict(score="softmax", groups=groups, keep=2, gscore="max")):
            check(torch_cuda, z, b, k=k, **kw)


def test_route_zero_tokens_and_graph_replay(torch_cuda):
    torch = torch_cuda
    import quantized_expert_ffn_bias_gb300 as coli
    d = _desc(coli, 256, 8, groups=8, keep=4)
    coli.colibri_moe_route(d, 0, None, 1, 256, None, None, None, None)
    z = torch.zeros((50, 256), device="cuda")
    idx, w = torch.zeros((50, 8), dtype=torch.int32, device="cuda"), torch.zeros((50, 8), device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        coli.colibri_moe_route(d, 50, z, 1, 256, None, idx, w, s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        coli.colibri_moe_route(d, 50, z, 1, 256, None, idx, w, torch.cuda.current_stream())
    rng = np.random.default_rng(3)
    for _ in range(2):
        zn = rng.standard_normal((50, 256)).astype(np.float32)
        z.copy_(torch.from_numpy(zn))
        g.replay()
        torch.cuda.synchronize()
        ids, ws = R.route(zn, None, k=8, groups=8, keep=4, scale=2.5)
        np.testing.assert_array_equal(idx.cpu().numpy(), ids)
        np.testing.assert_allclose(w.cpu().numpy(), ws, rtol=W_TOL)


@pytest.mark.parametrize("T", [1, 5, 8, 9, 40, 160])
@pytest.mark.parametrize("kind", ["groups", "softmax"])
def test_forward_with_a_set_routing(torch_cuda, T, kind):
    """The layer forward routes as the description says: its ids and weights match the 64-bit form of its own logits
    (away from near ties), its output is the oracle's for that choice, and None restores the plan's own routing bit for bit."""
    torch = torch_cuda
    import quantized_expert_ffn_bias_gb300 as coli
    from harness.device import DeviceLayer, to_dev
    layer = H.gen_layer(71, 0, d=512, F=256, E=32, k=4, rho=2.5, qtype=H.Q_INT4_G128, bias="uniform:0.1", F_shared=256)
    dl = DeviceLayer(layer, 160)
    x = H.gen_x(71, T, T, 512, H.X_BF16)
    xd = to_dev(x, dl.device)
    plain = dl.forward(xd).clone()
    kw = dict(groups=4, keep=2) if kind == "groups" else dict(score="softmax", renorm=False)
    dl.plan.set_route(_desc(coli, 32, 4, scale=1.75, **kw))
    out = dl.forward(xd)
    idx, w, nt, *_ = dl.routing(T)
    assert dl.plan.check_status(dl.ws) == 0
    xf = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).double().numpy()
    z = xf @ layer.router_w.astype(np.float64).T
    ids, ws = R.route(z, layer.bias, k=4, scale=1.75, **kw)
    toks = np.flatnonzero(nt == 0)
    assert len(toks) >= T - max(1, T // 20)
    np.testing.assert_array_equal(idx[toks], ids[toks])
    np.testing.assert_allclose(w[toks], ws[toks], rtol=2e-5)
    # the layer's output: every expert's result from the oracle, weighted by the choice
    y = combine(layer, xf, idx, w)
    check_output(out.cpu().numpy().astype(np.float64), y)
    dl.plan.set_route(None)
    assert torch.equal(dl.forward(xd), plain)
    dl.close()


def combine(layer, xf, idx, w):
    """Output of the layer for given ids and weights, in 64 bits: the oracle's experts one token at a time."""
    out = np.zeros(xf.shape)
    for t in range(xf.shape[0]):
        for j in range(idx.shape[1]):
            out[t] += float(w[t, j]) * O.expert_ffn(layer.experts, int(idx[t, j]), xf[t])
        if layer.shared is not None:
            out[t] += O.expert_ffn(layer.shared, 0, xf[t])
    return out


def test_set_routing_in_every_forward_call(torch_cuda):
    """The cached forward, the static-scratch forward and the pilot use the routing set on the plan; integer-dot inputs
    go with it."""
    torch = torch_cuda
    import quantized_expert_ffn_bias_gb300 as coli
    from harness.device import DeviceLayer, to_dev
    from tests.test_gpu_cache import pinned_bank
    layer = H.gen_layer(73, 0, d=512, F=256, E=32, k=4, rho=2.5, qtype=H.Q_INT4_G128, bias="uniform:0.1", F_shared=256)
    dl = DeviceLayer(layer, 12)
    st = torch.cuda.current_stream()
    keep, host = pinned_bank(torch, layer.experts)
    sb = coli.colibri_moe_cache_slot_bytes(dl.plan)
    slots = torch.empty(32 * sb, dtype=torch.uint8, device="cuda")
    cache = coli.Cache(dl.plan, 32, 1.0, host, slots, 32 * sb, shared=dl.shared.expert(0))
    ws = torch.empty(dl.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    for idot in (False, True):
        dl.plan.set_idot(idot)
        for T in (1, 3, 12):
            x = to_dev(H.gen_x(73, T, T, 512, H.X_BF16), dl.device)
            dl.plan.set_route(None)
            plain = dl.forward(x).clone()
            dl.plan.set_route(_desc(coli, 32, 4, score="softmax", groups=8, keep=2, gscore="max", scale=1.5))
            ref = dl.forward(x).clone()
            ids = dl.routing(T)[0]
            assert not torch.equal(ref, plain)
            out = torch.full_like(ref, float("nan"))
            cache.forward(T, x, dl.router_w, dl.bias, out, ws, stream=st)
            torch.cuda.synchronize()
            assert torch.equal(out, ref), "cached forward"
            out.fill_(float("nan"))
            dl.plan.forward_noalloc(T, x, dl.router_w, dl.bias, out, stream=st)
            torch.cuda.synchronize()
            assert torch.equal(out, ref), "forward with the static scratch"
            assert cache.pilot(T, x, dl.router_w, dl.bias, ws, stream=st) == sorted(set(ids.ravel().tolist()))
    torch.cuda.synchronize()
    cache.close()
    dl.close()
