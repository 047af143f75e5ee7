"""gq_ortho_step on every pair of tiles that a plan can take, against the
iteration in 64 bits.

Exact cases.  X holds 4^k entries of +-2^-k and zeros, so the norm is exact.
With the coefficients (3, -2, 256) and k = 5 or 6, G = X X^T, Q = -2 G + 256 G G
and 3 X + Q X are whole multiples of 2^(-2k), 2^(8-4k) and 2^(8-5k) and stay
below 2^24 of them (asserted for every matrix), so every binary32 sum is exact
in any order.  The results are then fixed to the bit by the roundings of what is
stored: G and Q in binary16 but for their diagonals, X in binary16 and, while
three steps or more are to come, 8 bits of what that leaves, and the output.
Steps with (1, 0, 0) before and behind, and one with (3, 0, 0) that shows the 8
bits, hand X on.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_ortho import COEF, _check, _plan_inputs, iterate

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
A, B, C = 3.0, -2.0, 256.0

# (tile of G and Q, of X): matrices, wide, tall, square and ragged; 64/64 on
# rings of four buffers with K whole, and in parts, and on two buffers
PLANS = [
    ((64, 64), [(70, 300), (301, 67), (129, 130)]),
    ((64, 64), [(100, 5000), (4100, 66)]),
    ((64, 64), [(150, 190), (190, 150), (135, 300)] * 34),
    ((64, 128), [(255, 1000), (1001, 250), (256, 512)] * 60),
    ((64, 256), [(500, 510), (510, 500), (490, 505)] * 40),
    ((128, 128), [(760, 768), (768, 761), (700, 767)] * 8),
    ((128, 256), [(1000, 1024), (1024, 1001)] * 8),
    ((256, 256), [(1000, 1020), (1024, 1000)] * 20 + [(1030, 700)] * 4),
]


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _sparse(gen, r, c):
    """(matrix of +-1 and zeros with 4^k entries, k)."""
    k = 6 if r * c >= 40000 else 5
    x = torch.zeros(r * c, device="cuda")
    at = torch.randperm(r * c, device="cuda", generator=gen)[:4 ** k]
    x[at] = torch.randint(0, 2, (4 ** k,), device="cuda", generator=gen).float() * 2 - 1
    return x.view(r, c), k


def _f32(v):
    """A sum that binary32 holds exactly (asserted)."""
    assert torch.equal(v.float().double(), v)
    return v.float()


def _want(x, k, out_mul, out):
    """The output that the exact sums and one rounding each give."""
    tr = x.shape[0] > x.shape[1]
    x = (x.t().contiguous() if tr else x).double() * 2.0 ** -k
    l = x.shape[1]
    scale = 2.0 ** float(np.round(0.5 * np.log2(np.float32(l))))
    g = _f32(x @ x.t().contiguous()).double()
    assert torch.equal(g.half().double(), g)        # (its diagonal is stored apart)
    q = _f32(B * g + C * (g @ g)).double()
    d = q.diagonal().clone()
    q = q.half().double()
    _f32(A + d)
    q.diagonal().copy_(d)
    new = _f32((A * x + q @ x) * scale)
    hi = new.half()
    low = ((new - hi.float()) * 2.0 ** 14).clamp(-448, 448).to(torch.float8_e4m3fn)
    new = _f32(hi.double() + low.double() * 2.0 ** -14).double()
    new = _f32(3 * new).half().double()
    res = _f32(new / scale * out_mul).to(TORCH[out])
    return res.t().contiguous() if tr else res


@pytest.mark.parametrize("n", range(len(PLANS)))
def test_every_tile_exactly(gq, n):
    tiles, shapes = PLANS[n]
    gen = torch.Generator(device="cuda").manual_seed(n)
    # 64 out: the smallest entries stay normal in binary16
    mul = [64.0 * (1 + i % 2) for i in range(len(shapes))]
    coef = [(1, 0, 0), (A, B, C), (3, 0, 0), (1, 0, 0), (1, 0, 0)]
    for gap, dt, out, mom, nesterov in ((0, "f32", "bf16", True, True), (3, "f16", "f16", False, False),
                                        (8, "bf16", "f16", True, False), (4, "f32", "f16", False, True)):
        say("tiles", tiles, len(shapes), "matrices, gap", gap, dt, out, mom, nesterov)
        off, total = _plan_inputs(shapes, gap)
        g = torch.full((total,), float("nan"), device="cuda")
        xs = []
        for o, (r, c) in zip(off, shapes):
            xs.append(_sparse(gen, r, c))
            g[o:o + r * c] = xs[-1][0].reshape(-1) * 0.25
        g = g.to(TORCH[dt])
        m = torch.full((total,), float("nan"), device="cuda") if mom else None
        res = torch.full((total,), 77.0, dtype=TORCH[out], device="cuda")
        plan = gq.gq_ortho_create(shapes, off, steps=5, coef=coef, eps=0.0, out_mul=mul)
        assert gq.gq_ortho_tiles(plan) == tiles
        for again in range(2):          # the plan's workspace is used again
            if mom:
                for o, (r, c) in zip(off, shapes):
                    m[o:o + r * c] = 0.0
            res.fill_(77.0)
            gq.gq_ortho_step(plan, g, res, in_mul=0.5, momentum=m, mu=1.0, nesterov=nesterov)
            inside = torch.zeros(total, dtype=torch.bool, device="cuda")
            for i, (o, (r, c)) in enumerate(zip(off, shapes)):
                want = _want(*xs[i], mul[i], out)
                got = res[o:o + r * c].view(r, c)
                assert torch.equal(got, want), (i, r, c, (got != want).nonzero()[:3].tolist())
                if mom:
                    assert torch.equal(m[o:o + r * c], xs[i][0].reshape(-1) * 0.125)
                inside[o:o + r * c] = True
            assert bool((res[~inside] == 77.0).all()), "wrote between the matrices"
            if mom:
                assert bool(torch.isnan(m[~inside]).all()), "wrote between the momenta"
        plan.close()


@pytest.mark.parametrize("n", range(len(PLANS)))
def test_every_tile_within_the_bound(gq, n):
    """The default iteration on dense gradients; equal matrices, wherever they
    lie, give equal bits."""
    tiles, shapes = PLANS[n]
    rng = np.random.default_rng(n)
    first = {}
    for s in shapes:
        if s not in first:
            p = rng.standard_normal((s[0], 5)) @ rng.standard_normal((5, s[1]))
            first[s] = ((0.2 * p + rng.standard_normal(s)) * 1e-3).astype(np.float32)
    off, total = _plan_inputs(shapes, 5)
    g = torch.zeros(total, device="cuda")
    for o, s in zip(off, shapes):
        g[o:o + s[0] * s[1]] = torch.from_numpy(first[s].reshape(-1)).cuda()
    g = g.half() if n % 2 else g
    res = torch.zeros(total, dtype=torch.float16, device="cuda")
    plan = gq.gq_ortho_create(shapes, off)
    assert gq.gq_ortho_tiles(plan) == tiles
    gq.gq_ortho_step(plan, g, res)
    one = {}
    for o, s in zip(off, shapes):
        got = res[o:o + s[0] * s[1]]
        if s not in one:
            one[s] = got
            u = g[o:o + s[0] * s[1]].double().cpu().numpy().reshape(s)
            want, bound = iterate(u, [COEF] * 5)
            rel = _check(got.double().cpu().numpy().reshape(s), want, bound, "f16")
            say(tiles, s, "rel %.2e" % rel)
        assert torch.equal(got, one[s]), (tiles, s)
    plan.close()


def test_one_work_group_plans_have_no_tiles(gq):
    plan = gq.gq_ortho_create([(64, 256), (200, 63)])
    assert gq.gq_ortho_tiles(plan) == (0, 0)
    plan.close()
