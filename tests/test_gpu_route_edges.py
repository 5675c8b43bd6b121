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
