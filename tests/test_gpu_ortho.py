"""gq_ortho_step on the GPU against the iteration in 64 bits.

Tolerance.  With phi(s) = a s + b s^3 + c s^5 a step maps X = U S V^T to
U phi(S) V^T.  To first order an error E of X becomes one of at most L |E|_F,
L the largest of |phi(si) - phi(sj)| / |si - sj|, |phi(si) + phi(sj)| / (si +
sj), |phi'(si)| and, for a matrix that is not square, |phi(si) / si|, over the
singular values (for a square or a wide matrix these are all the factors of
the derivative of an odd matrix function).  A step adds, with h = 2^-11 (half
a step of binary16) and t = K 2^-24 for a binary32 sum of K terms:
  dG = h |G| + t | |X| |X|^T |                          (Frobenius norms)
  dQ = |b| dG + 2 |c| |G|_2 dG + t |c| | |G| |G| | + h |Q|
  dX = dQ |X|_2 + t | |Q| |X| | + h |X'|
and each stored entry at most 2^-25 more where it is subnormal.  The bound is
the sum of the steps' dX, each grown by the following steps' L, and half a
step of the output's type; 1.2 times that covers the second order."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
COEF = (3.4445, -4.7750, 2.0315)
H = 2.0 ** -11


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _fro(x):
    return float(np.linalg.norm(x))


def iterate(u, coefs, eps=1e-7):
    """(X, bound on the kernel's distance from it) in 64 bits."""
    tr = u.shape[0] > u.shape[1]
    x = (u.T if tr else u) / (_fro(u) + eps)
    s, l = x.shape
    sub = np.sqrt(s * l) * 2.0 ** -25 / 2.0 ** np.round(0.5 * np.log2(l))
    err = H * _fro(x) + sub
    for a, b, c in coefs:
        sig = np.linalg.svd(x, compute_uv=False)
        phi = a * sig + b * sig ** 3 + c * sig ** 5
        slope = np.abs(a + 3 * b * sig ** 2 + 5 * c * sig ** 4)
        d = np.abs(sig[:, None] - sig)
        div = np.abs(phi[:, None] - phi) / np.where(d > 1e-9, d, np.inf)
        add = np.abs(phi[:, None] + phi) / np.maximum(sig[:, None] + sig, 1e-300)
        add[sig[:, None] + sig == 0] = abs(a)
        L = max(slope.max(), div.max(), add.max())
        g = x @ x.T
        q = b * g + c * g @ g
        t_l, t_s = l * 2.0 ** -24, s * 2.0 ** -24
        dg = H * _fro(g) + t_l * _fro(np.abs(x) @ np.abs(x).T) + s * 2.0 ** -25
        dq = (abs(b) + 2 * abs(c) * np.linalg.norm(g, 2)) * dg + H * _fro(q) + s * 2.0 ** -25
        dq += t_s * abs(c) * _fro(np.abs(g) @ np.abs(g))
        new = a * x + q @ x
        dx = dq * sig[0] + t_s * _fro(np.abs(q) @ np.abs(x)) + H * _fro(new) + sub
        err = L * err + dx
        x = new
    return (x.T if tr else x), 1.2 * err


def _gradients(rng, shapes, kind):
    parts = []
    for r, c in shapes:
        g = rng.standard_normal((r, c))
        if kind == "low":
            p = min(3, r, c)
            g = 0.1 * g + rng.standard_normal((r, p)) @ rng.standard_normal((p, c))
        elif kind == "eye":
            g = np.zeros((r, c))
            np.fill_diagonal(g, rng.choice([-1.0, 1.0], min(r, c)))
            g = g[rng.permutation(r)]
        parts.append((g * 1e-3).astype(np.float32))
    return parts


SHAPES = [[(1, 1)], [(1, 7), (7, 1), (5, 5)], [(64, 147)], [(1000, 64), (33, 1024), (64, 64)],
          [(64, 256), (200, 63)], [(64, 1025)], [(65, 300)], [(40, 5000)], [(4100, 130), (70, 2100)], [(147, 64), (64, 64), (65, 63)],
          [(31, 200), (200, 31), (129, 129), (100, 1000)], [(300, 700), (700, 300)],
          [(256, 512)] * 3, [(1024, 1100), (1030, 1000)]]


def _plan_inputs(shapes, gap):
    off, at = [], gap
    for r, c in shapes:
        off.append(at)
        at += r * c + gap
    return np.array(off), at


def _check(got, want, bound, out):
    half = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[out]
    tol = bound + half * _fro(want) + 2.0 ** -25 * np.sqrt(want.size)
    d = _fro(got - want)
    assert d <= tol, (d, tol, _fro(want))
    return d / max(_fro(want), 1e-300)


@pytest.mark.parametrize("dt,out", [("f32", "bf16"), ("f16", "f16"), ("bf16", "f16")])
@pytest.mark.parametrize("kind", ["noise", "low", "eye"])
def test_step(gq, dt, out, kind):
    rng = np.random.default_rng(4)
    for shapes in SHAPES:
        for gap, mul in ((0, 1.0), (3, 2.0 ** -10)):
            off, n = _plan_inputs(shapes, gap)
            say("ortho", dt, out, kind, shapes, "gap", gap)
            parts = _gradients(rng, shapes, kind)
            flat = np.zeros(n, np.float32)
            for o, g in zip(off, parts):
                flat[o:o + g.size] = g.reshape(-1) / np.float32(mul)
            g = torch.from_numpy(flat).to(TORCH[dt]).cuda()
            res = torch.full((n,), 77.0, dtype=TORCH[out], device="cuda")
            plan = gq.gq_ortho_create(shapes, off)
            gq.gq_ortho_step(plan, g, res, in_mul=mul)
            r = res.double().cpu().numpy()
            v = g.double().cpu().numpy() * mul
            seen = np.zeros(n, bool)
            for o, (rows, cols) in zip(off, shapes):
                want, bound = iterate(v[o:o + rows * cols].reshape(rows, cols), [COEF] * 5)
                rel = _check(r[o:o + rows * cols].reshape(rows, cols), want, bound, out)
                say("  ", rows, cols, "rel %.2e" % rel)
                seen[o:o + rows * cols] = True
            assert np.all(r[~seen] == 77.0), "wrote between the matrices"
            plan.close()


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_momentum(gq, nesterov, dt):
    """Momentum is two rounded binary32 operations: exact bits, over steps."""
    rng = np.random.default_rng(6)
    shapes = [(33, 70), (70, 33), (64, 64), (1, 5)]
    off, n = _plan_inputs(shapes, 1)
    mu, mul = np.float32(0.95), np.float32(2.0 ** -6)
    m = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    ref = m.cpu().numpy().copy()
    plan = gq.gq_ortho_create(shapes, off)
    res = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    inside = np.zeros(n, bool)
    for o, (r, c) in zip(off, shapes):
        inside[o:o + r * c] = True
    for _ in range(3):
        g = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(TORCH[dt]).cuda()
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


def test_steps_and_coefficients(gq):
    """Other step counts and coefficients (1 to 16 steps of the cubic
    iteration 1.5 x - 0.5 x^3, whose singular values rise to 1)."""
    rng = np.random.default_rng(7)
    u = rng.standard_normal((40, 90)).astype(np.float32)
    g = torch.from_numpy(u.reshape(-1)).cuda()
    for steps in (1, 2, 3, 16):
        coef = [(1.5, -0.5, 0.0)] * steps
        plan = gq.gq_ortho_create([(40, 90)], steps=steps, coef=coef, eps=0.0, out_mul=[0.25])
        res = torch.zeros(u.size, dtype=torch.float16, device="cuda")
        gq.gq_ortho_step(plan, g, res)
        want, bound = iterate(u.astype(np.float64), coef, 0.0)
        _check(4 * res.double().cpu().numpy().reshape(u.shape), want, bound, "f16")
        if steps == 16:
            r = 4 * res.double().cpu().numpy().reshape(u.shape)
            assert np.abs(r @ r.T - np.eye(40)).max() < 0.01


def test_zero_and_not_finite(gq):
    shapes = [(20, 30), (70, 20), (64, 64), (30, 20)]
    off, n = _plan_inputs(shapes, 0)
    rng = np.random.default_rng(8)
    flat = rng.standard_normal(n).astype(np.float32)
    flat[:600] = 0.0
    flat[off[1] + 5] = np.inf
    flat[off[3] + 7] = np.nan
    clean = flat.copy()
    clean[off[1]:off[2]] = 1.0
    clean[off[3]:] = 1.0
    plan = gq.gq_ortho_create(shapes)
    res = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    gq.gq_ortho_step(plan, torch.from_numpy(flat).cuda(), res[0])
    gq.gq_ortho_step(plan, torch.from_numpy(clean).cuda(), res[1])
    fresh = gq.gq_ortho_create(shapes)
    gq.gq_ortho_step(fresh, torch.from_numpy(clean).cuda(), res[2])
    a, b = off[1], off[2]
    assert bool((res[0][:600] == 0).all())
    assert bool(torch.isnan(res[0][a:b]).all()) and bool(torch.isnan(res[0][off[3]:]).all())
    assert torch.equal(res[0][b:off[3]], res[1][b:off[3]])
    # a plan that has seen them gives what a fresh one gives
    assert torch.equal(res[1], res[2]) and bool(torch.isfinite(res[1]).all())


def test_sizes_of_gradients(gq):
    """The norm neither overflows nor vanishes: gradients of 1e-39 (subnormal)
    to 1e30."""
    rng = np.random.default_rng(9)
    u = rng.standard_normal((48, 80))
    plan = gq.gq_ortho_create([(48, 80)], eps=0.0)
    for size in (1e-39, 1e-30, 1.0, 1e30):
        g = torch.from_numpy((u * size).astype(np.float32).reshape(-1)).cuda()
        res = torch.zeros(u.size, dtype=torch.float16, device="cuda")
        gq.gq_ortho_step(plan, g, res)
        want, bound = iterate(g.double().cpu().numpy().reshape(u.shape), [COEF] * 5, 0.0)
        _check(res.double().cpu().numpy().reshape(u.shape), want, bound, "f16")


def test_reduce_then_step_run(gq):
    """Gradients quantized, reduced in rank order and orthogonalised, on a
    stream of their own, then captured and replayed."""
    rng = np.random.default_rng(11)
    shapes = [(96, 64), (64, 200), (33, 65)]
    off, n = _plan_inputs(shapes, 0)
    W = 3
    xs = [torch.from_numpy(rng.standard_normal(n).astype(np.float32) * 1e-3).cuda()
          for _ in range(W)]
    units = gq.gq_units_create(np.concatenate([off, [n]]))
    U = len(shapes)
    scales = [torch.empty(U, device="cuda") for _ in range(W)]
    codes = [torch.empty(n, dtype=torch.int8, device="cuda") for _ in range(W)]
    so, qo = torch.empty(U, device="cuda"), torch.empty(n, dtype=torch.int8, device="cuda")
    r, m = torch.empty(n, device="cuda"), torch.zeros(n, device="cuda")
    out = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    plan = gq.gq_ortho_create(shapes)

    def step():
        gq.gq_quantize(xs, units, scales, codes)
        gq.gq_reduce_requantize(codes, scales, units, so, qo, r_out=r)
        gq.gq_ortho_step(plan, r, out, in_mul=1.0 / W, momentum=m, mu=0.9, nesterov=True)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = r.cpu().numpy() * np.float32(1.0 / W)
    mm = g.copy()
    u = (g + np.float32(0.9) * mm).astype(np.float64)
    got = out.double().cpu().numpy()
    for o, (rows, cols) in zip(off, shapes):
        want, bound = iterate(u[o:o + rows * cols].reshape(rows, cols), [COEF] * 5)
        _check(got[o:o + rows * cols].reshape(rows, cols), want, bound, "bf16")
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        m.zero_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first), i
        m.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, first), i


def test_zero_without_eps(gq):
    """A zero matrix gives 0 with eps = 0 too, and leaves the others alone."""
    rng = np.random.default_rng(15)
    for shapes in ([(20, 30), (30, 20), (5, 5)], [(70, 300), (300, 70), (65, 65)]):
        off, n = _plan_inputs(shapes, 0)
        flat = rng.standard_normal(n).astype(np.float32)
        flat[:off[1]] = 0.0
        plan = gq.gq_ortho_create(shapes, eps=0.0)
        res = torch.full((n,), 7.0, dtype=torch.float16, device="cuda")
        gq.gq_ortho_step(plan, torch.from_numpy(flat).cuda(), res)
        assert bool((res[:off[1]] == 0).all())
        for o, (r, c) in list(zip(off, shapes))[1:]:
            want, bound = iterate(flat[o:o + r * c].reshape(r, c).astype(np.float64), [COEF] * 5, 0.0)
            _check(res[o:o + r * c].double().cpu().numpy().reshape(r, c), want, bound, "f16")


def test_many_matrices_far_apart(gq):
    """Hundreds of small matrices of few rows, and one whose elements lie
    above 2^32 in the flat buffers."""
    rng = np.random.default_rng(16)
    shapes = [(64, 300)] * 150 + [(1, 400)] * 150 + [(90, 40)]
    off, n = _plan_inputs(shapes, 0)
    off[-1] += 1 << 32
    n += 1 << 32
    parts = [(rng.standard_normal(s) * 1e-3).astype(np.float32) for s in shapes]
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    for o, p in zip(off, parts):
        g[o:o + p.size] = torch.from_numpy(p.reshape(-1)).cuda()
    plan = gq.gq_ortho_create(shapes, off)
    assert gq.gq_ortho_info(plan)["n"] == n
    res = torch.full((n,), 7.0, dtype=torch.bfloat16, device="cuda")
    gq.gq_ortho_step(plan, g, res)
    for i in (0, 77, 149, 150, 151, 299, 300):
        o, (r, c) = off[i], shapes[i]
        say("matrix", i, r, c, "at", int(o))
        u = g[o:o + r * c].double().cpu().numpy().reshape(r, c)
        want, bound = iterate(u, [COEF] * 5)
        _check(res[o:o + r * c].double().cpu().numpy().reshape(r, c), want, bound, "bf16")
    end = off[-2] + 400
    assert bool((res[end:end + (1 << 20)] == 7).all()) and bool((res[off[-1] - 1000:off[-1]] == 7).all())
