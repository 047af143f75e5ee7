"""What gq_ortho_step promises beside the iteration, on plans whose matrices
are too large for one work group: momentum to the bit, numbers of steps and
coefficients, zero, infinite and NaN matrices, extreme norms, captured and
replayed calls, and a training step's whole run.  Tolerances: those of
tests/test_gpu_ortho.py."""
import pathlib
import re

import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_ortho import COEF, _check, _plan_inputs, iterate

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SHAPES = [(70, 300), (301, 67), (129, 1030), (5, 7), (66, 66)]


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _tiled(gq, plan):
    assert min(gq.gq_ortho_tiles(plan)) >= 64
    return plan


@pytest.mark.parametrize("gap", [0, 1, 4, 8])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_momentum(gq, dt, nesterov, gap):
    """Two rounded binary32 operations: exact bits, over steps, at starts and
    rows of every alignment."""
    rng = np.random.default_rng(31)
    shapes = SHAPES + ([(72, 304), (304, 72), (68, 300)] if gap % 4 == 0 else [])
    off, n = _plan_inputs(shapes, gap)
    mu, mul = np.float32(0.95), np.float32(2.0 ** -6)
    m = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    ref = m.cpu().numpy().copy()
    plan = _tiled(gq, gq.gq_ortho_create(shapes, off))
    res = torch.full((n,), 7.0, dtype=torch.bfloat16, device="cuda")
    inside = np.zeros(n, bool)
    for o, (r, c) in zip(off, shapes):
        inside[o:o + r * c] = True
    for step in range(2):
        g = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(TORCH[dt]).cuda()
        say("momentum", dt, nesterov, "gap", gap, "step", step)
        gq.gq_ortho_step(plan, g, res, in_mul=float(mul), momentum=m, mu=float(mu),
                         nesterov=nesterov)
        gf = g.float().cpu().numpy() * mul
        ref[inside] = (mu * ref + gf)[inside]
        assert np.array_equal(m.cpu().numpy().view(np.uint32), ref.view(np.uint32))
        u = (gf + mu * ref if nesterov else ref).astype(np.float64)
        r = res.double().cpu().numpy()
        for o, (rows, cols) in zip(off, shapes):
            want, bound = iterate(u[o:o + rows * cols].reshape(rows, cols), [COEF] * 5)
            _check(r[o:o + rows * cols].reshape(rows, cols), want, bound, "bf16")
        assert np.all(r[~inside] == 7.0), "wrote between the matrices"


@pytest.mark.parametrize("steps", [1, 2, 3, 16])
def test_steps_and_coefficients(gq, steps):
    """The cubic iteration 1.5 x - 0.5 x^3 and one whose coefficients differ
    from step to step; a factor of each matrix of its own."""
    rng = np.random.default_rng(32)
    off, n = _plan_inputs(SHAPES, 3)
    flat = rng.standard_normal(n).astype(np.float32)
    mul = [0.25, 2.0, -1.0, 0.5, 8.0]
    for coef in ([(1.5, -0.5, 0.0)] * steps,
                 [(1.5 + 0.25 * (k % 3), -0.5 - 0.125 * (k % 2), 0.0625 * (k % 4)) for k in range(min(steps, 3))]
                 + [(1.5, -0.5, 0.0)] * max(0, steps - 3)):
        say("steps", steps, coef[:3])
        plan = _tiled(gq, gq.gq_ortho_create(SHAPES, off, steps=steps, coef=coef, eps=0.0, out_mul=mul))
        res = torch.zeros(n, dtype=torch.float16, device="cuda")
        gq.gq_ortho_step(plan, torch.from_numpy(flat).cuda(), res)
        for o, (r, c), f in zip(off, SHAPES, mul):
            want, bound = iterate(flat[o:o + r * c].reshape(r, c).astype(np.float64), coef, 0.0)
            got = res[o:o + r * c].double().cpu().numpy().reshape(r, c) / f
            # (powers of two: the quotient is exact, and so is its rounding's size)
            _check(got, want, bound, "f16")


def test_zero_and_not_finite(gq):
    shapes = [(70, 300), (301, 67), (129, 1030), (66, 66), (100, 90)]
    off, n = _plan_inputs(shapes, 0)
    rng = np.random.default_rng(33)
    flat = rng.standard_normal(n).astype(np.float32)
    size = [r * c for r, c in shapes]
    flat[off[0]:off[0] + size[0]] = 0.0
    flat[off[1] + 5] = np.inf
    flat[off[3] + size[3] - 1] = np.nan
    clean = flat.copy()
    for i in (1, 3):
        clean[off[i]:off[i] + size[i]] = rng.standard_normal(size[i])
    for eps in (1e-7, 0.0):
        plan = _tiled(gq, gq.gq_ortho_create(shapes, eps=eps))
        fresh = gq.gq_ortho_create(shapes, eps=eps)
        for mom in (False, True):
            res = [torch.full((n,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
            for p, v, o in ((plan, flat, res[0]), (plan, clean, res[1]), (fresh, clean, res[2])):
                m = torch.zeros(n, device="cuda") if mom else None
                gq.gq_ortho_step(p, torch.from_numpy(v).cuda(), o, momentum=m)
            part = [[o[off[i]:off[i] + size[i]] for i in range(5)] for o in res]
            assert bool((part[0][0] == 0).all())
            assert bool(torch.isnan(part[0][1]).all()) and bool(torch.isnan(part[0][3]).all())
            for i in (2, 4):
                assert torch.equal(part[0][i], part[1][i]), i
            # a plan that has seen them gives what a fresh one gives
            assert torch.equal(res[1], res[2]) and bool(torch.isfinite(res[1]).all())


def test_sizes_of_gradients(gq):
    """The norm neither overflows nor vanishes: gradients of 1e-39 (subnormal)
    to 1e30, with and without momentum."""
    rng = np.random.default_rng(34)
    u = rng.standard_normal((90, 280))
    plan = _tiled(gq, gq.gq_ortho_create([(90, 280)], eps=0.0))
    for size in (1e-39, 1e-30, 1.0, 1e30):
        for mom in (False, True):
            g = torch.from_numpy((u * size).astype(np.float32).reshape(-1)).cuda()
            res = torch.zeros(u.size, dtype=torch.float16, device="cuda")
            m = torch.zeros(u.size, device="cuda") if mom else None
            gq.gq_ortho_step(plan, g, res, momentum=m, mu=0.5, nesterov=False)
            want, bound = iterate(g.double().cpu().numpy().reshape(u.shape), [COEF] * 5, 0.0)
            _check(res.double().cpu().numpy().reshape(u.shape), want, bound, "f16")


@pytest.mark.parametrize("shapes", [SHAPES, [(100, 5000), (70, 66)],
                                    [(255, 1000), (1001, 250), (256, 512)] * 60])
def test_replayed_with_reduced_gradients(gq, shapes):
    """Quantized, reduced in rank order and orthogonalised on a stream of its
    own, then captured, replayed and mixed with eager calls of the same plan,
    which its order of K splits or not."""
    gen = torch.Generator(device="cuda").manual_seed(35)
    off, n = _plan_inputs(shapes, 0)
    W = 2
    xs = [torch.randn(n, device="cuda", generator=gen) * 1e-3 for _ in range(W)]
    units = gq.gq_units_create(np.concatenate([off, [n]]))
    U = len(shapes)
    scales = [torch.empty(U, device="cuda") for _ in range(W)]
    codes = [torch.empty(n, dtype=torch.int8, device="cuda") for _ in range(W)]
    so, qo = torch.empty(U, device="cuda"), torch.empty(n, dtype=torch.int8, device="cuda")
    r, m = torch.empty(n, device="cuda"), torch.zeros(n, device="cuda")
    out = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    plan = _tiled(gq, gq.gq_ortho_create(shapes))

    def step():
        gq.gq_quantize(xs, units, scales, codes)
        gq.gq_reduce_requantize(codes, scales, units, so, qo, r_out=r)
        gq.gq_ortho_step(plan, r, out, in_mul=1.0 / W, momentum=m, mu=0.9)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = r.cpu().numpy() * np.float32(1.0 / W)
    u = (g + np.float32(0.9) * g).astype(np.float64)
    got = out.double().cpu().numpy()
    for o, (rows, cols) in list(zip(off, shapes))[:3]:
        want, bound = iterate(u[o:o + rows * cols].reshape(rows, cols), [COEF] * 5)
        _check(got[o:o + rows * cols].reshape(rows, cols), want, bound, "bf16")
    first, mfirst = out.clone(), m.clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]      # of one plan, run in order
    for graph in graphs:
        with torch.cuda.graph(graph):
            step()
    for i in range(3):
        for run in (graphs[0].replay, step, graphs[1].replay):
            m.zero_()
            out.zero_()
            run()
            torch.cuda.synchronize()
            assert torch.equal(out, first) and torch.equal(m, mfirst), i


def test_readme_update_value(gq):
    """The README's training step: its update is that of the summed gradient."""
    text = (pathlib.Path(__file__).resolve().parent.parent / "README.md").read_text()
    program = [p for p in re.findall(r"```python\n(.*?)```", text, re.S) if "gq_ortho_step" in p]
    names = {"torch": torch, "gq": gq}
    exec(program[0], names)
    torch.cuda.synchronize()
    assert min(gq.gq_ortho_tiles(names["plan"])) >= 64
    g = names["total"].cpu().numpy() * np.float32(1.0 / names["W"])
    assert np.array_equal(names["momentum"].cpu().numpy(), g)
    shape = (names["m"], names["k"])
    u = (g + np.float32(0.95) * g).astype(np.float64).reshape(shape)
    want, bound = iterate(u, [COEF] * 5)
    rel = _check(names["update"].double().cpu().numpy().reshape(shape), want, bound, "bf16")
    say("README update rel %.2e" % rel)
