"""Routing from given logits at the edges of its arithmetic (needs a GB300): borders inside the buckets of its cut scores,
and chosen scores below fp32's range."""
from __future__ import annotations

import numpy as np
import pytest

from tests import serving_ref as R
from tests.test_gpu_route import check, torch_cuda  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [128, 256, 384, 512, 1024])
def test_route_clusters_wider_than_the_scores_error(torch_cuda, E):
    """Logits within 300 to 5,000 fp32 steps of one another, so that some are certainly above the last pick, some certainly
    below and some between, in every order of ids."""
    rng = np.random.default_rng(E)
    T = 160
    base = rng.choice(np.array([0.5, -2.0, 0.03], np.float32), (T, 1))
    width = rng.choice(np.array([300, 1000, 3000, 5000]), (T, 1))
    z = (base + (rng.random((T, E)) * 2 - 1) * width * np.spacing(np.abs(base))).astype(np.float32)
    for k in (1, 8, 32):
        check(torch_cuda, z, None, k=k)
        check(torch_cuda, z, np.full(E, -0.125, np.float32), k=k)
        check(torch_cuda, z, None, k=k, score="softmax", renorm=False)
        check(torch_cuda, z, None, k=min(k, E // 16 * 3), groups=16, keep=3, gscore="max")
        check(torch_cuda, z, None, k=min(k, E // 16 * 3), groups=16, keep=3, gscore="top2")


@pytest.mark.parametrize("E", [128, 256, 384, 512, 1024])
def test_route_border_inside_a_bucket(torch_cuda, E):
    """Two experts side by side at every distance above the last pick, the lower id with the lower score: one may be
    certain and the other not.  Each of the three best is chosen, none twice (the last pick's id lies between the two, so that no
    entry keeps the value of an earlier pass)."""
    for top in (0.6, 0.7, 0.85):
        a = np.float32(top).view(np.int32) & ~31
        for d in range(1, 130):
            for gap in (1, 2):
                u = np.full(E, -1.0, np.float32)
                for e, off in ((50, 0), (60, -1), (10, d), (100, d + gap)):
                    u[e] = np.int32(a + off).view(np.float32)
                check(torch_cuda, np.zeros((1, E), np.float32), u - np.float32(0.5), k=3)


@pytest.mark.parametrize("level", [-70.0, -100.0, -300.0, -700.0])
def test_route_renormalised_weights_of_tiny_scores(torch_cuda, level):
    """Every chosen score is below fp32's range (or close to it); their ratios are not."""
    rng = np.random.default_rng(int(-level))
    z = (level + rng.uniform(-3, 3, (40, 64))).astype(np.float32)
    check(torch_cuda, z, None, k=6)
    check(torch_cuda, z, None, k=6, groups=8, keep=3)
    bias = (rng.standard_normal(64) * 0.1).astype(np.float32)
    check(torch_cuda, z, bias, k=6)
    # softmax: logits far above all others, shut out by their biases or by their group
    z2 = (rng.uniform(-3, 3, (40, 64))).astype(np.float32)
    z2[:, 7] = -level
    shut = np.zeros(64, np.float32)
    shut[7] = -np.inf
    check(torch_cuda, z2, shut, k=6, score="softmax")
    forced = np.zeros(64, np.float32)
    forced[16:32] = 2.0
    check(torch_cuda, z2, forced, k=6, score="softmax", groups=4, keep=1, gscore="max")
    check(torch_cuda, z2, forced, k=6, score="softmax", renorm=False, groups=4, keep=1, gscore="max")


def test_route_weights_without_any_score(torch_cuda):
    """Scores of 0 in 64 bits: the weights are 0."""
    z = np.full((3, 64), -np.inf, np.float32)
    z[1] = np.finfo(np.float32).min
    z[2] = -2000.0
    check(torch_cuda, z, None, k=6)
    z[:, 0] = 1.0
    shut = np.zeros(64, np.float32)
    shut[0] = -np.inf
    check(torch_cuda, z, shut, k=6)
    check(torch_cuda, z, shut, k=6, score="softmax")
    z[:, 0] = np.inf
    check(torch_cuda, z, shut, k=6, score="softmax")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_scores_around_the_smallest_normal_number(torch_cuda, score):
    """Scores of 2^-120 to 2^-132, of which fp32 arithmetic may flush any below 2^-126 to 0: in sums of two they decide
    between groups, with biases as small between experts."""
    rng = np.random.default_rng(126)
    for E, groups in ((64, 8), (256, 8), (384, 6), (62, 31)):
        z = rng.uniform(-91.5, -86.0, (300, E)).astype(np.float32)
        if score == "softmax":
            z[:, 3] = 0.0                              # the sum is 1, the others' scores are exp(z)
        shut = np.zeros(E, np.float32)
        shut[3] = -np.inf
        small = (rng.standard_normal(E) * 2.0 ** -126).astype(np.float32)
        small[3] = -np.inf
        keep = max(2, groups // 3)
        for bias in (shut, small):
            check(torch_cuda, z, bias, k=4, score=score, renorm=False)
            check(torch_cuda, z, bias, k=4, score=score)
            for gscore in ("top2", "max"):
                check(torch_cuda, z, bias, k=4, score=score, groups=groups, keep=keep, gscore=gscore)
