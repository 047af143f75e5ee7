"""X = u / (|u| + eps) is rounded to binary16 once: quotients that lie closer to
the middle of two values than a binary32 number can tell."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _eps(j):
    """A binary32 eps that takes 1 / (1 + eps) to within 2^-30 of the middle
    1 - (2 j + 1) 2^-12 of two binary16 values, and the nearer one of them."""
    mid = 1 - Fraction(2 * j + 1, 4096)
    eps = np.float32(float(1 / mid - 1))
    x = 1 / (1 + Fraction(float(eps)))
    assert 0 < abs(x - mid) < Fraction(1, 1 << 30) and np.float32(float(x)) == np.float32(float(mid))
    return float(eps), float(mid + Fraction(1 if x > mid else -1, 4096))


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("momentum", [False, True])
def test_x_is_rounded_once(gq, tiled, momentum):
    shapes = [(1, 1), (1, 4), (4, 1)] + ([(65, 300)] if tiled else [])
    n = sum(r * c for r, c in shapes)
    g = torch.zeros(n, device="cuda")
    g[0] = g[1] = g[5] = 1.0        # the first element of each small matrix
    wants = [_eps(j) for j in range(24)]
    # both sides of the middle, and both kinds of neighbours, are among them
    assert len({(w > 1 - (2 * j + 1) / 4096, j % 2) for j, (_, w) in enumerate(wants)}) == 4
    for eps, want in wants:
        plan = gq.gq_ortho_create(shapes, steps=1, coef=[(1, 0, 0)], eps=eps)
        assert (min(gq.gq_ortho_tiles(plan)) > 0) == tiled
        out = torch.full((n,), 7.0, dtype=torch.float16, device="cuda")
        m = torch.zeros(n, device="cuda") if momentum else None
        gq.gq_ortho_step(plan, g, out, momentum=m, mu=0.0)
        got = out.double().cpu().numpy()
        assert got[0] == got[1] == got[5] == want, (eps, got[[0, 1, 5]], want)
        got[[0, 1, 5]] = 0
        assert not got.any()
        plan.close()
