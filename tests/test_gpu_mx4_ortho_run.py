"""The 4-bit exchange and the orthogonalised update as a training step uses
them together: weight gradients of two matrices from 4-bit activations into one
flat gradient, its exchange between ranks in 4 bits, and the update; on a
stream of its own, then captured and replayed.  And the README's programs."""
import pathlib
import re

import numpy as np
import pytest
import torch

from tests import mx4_ref as ref
from tests.test_gpu_ortho import COEF, _check, iterate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def test_step_from_activations_to_update(gq):
    rng = np.random.default_rng(21)
    T, W = 2100, 2
    shapes = [(70, 45), (33, 200)]      # outputs x inputs of two layers
    off = np.concatenate([[0], np.cumsum([m * k for m, k in shapes])])
    n = int(off[-1])

    def buf(k):
        return torch.empty(k, dtype=torch.uint8, device="cuda")

    def act(cols):
        return torch.from_numpy(rng.standard_normal((T, cols)).astype(np.float32)).bfloat16().cuda()

    acts = [[(act(m), act(k)) for m, k in shapes] for _ in range(W)]
    work = []
    for m, k in shapes:
        (ny, by), (nx, bx) = gq.gq_mx4_sizes(m, T), gq.gq_mx4_sizes(k, T)
        work.append((buf(ny), buf(by), buf(nx), buf(bx), buf(gq.gq_mx4_product_workspace(m, k, T))))
    grad = [torch.zeros(n, device="cuda") for _ in range(W)]
    ng, bg = gq.gq_mx4_sizes(1, n)
    sg, qg = [buf(ng) for _ in range(W)], [buf(bg) for _ in range(W)]
    total, momentum = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    update = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    plan = gq.gq_ortho_create(shapes, off[:-1])

    def step():
        for w in range(W):
            for i, (m, k) in enumerate(shapes):
                sy, qy, sx, qx, ws = work[i]
                gq.gq_mx4_quantize([acts[w][i][0]], [sy], [qy], transpose=True)
                gq.gq_mx4_quantize([acts[w][i][1]], [sx], [qx], transpose=True)
                gq.gq_mx4_product(qy, sy, qx, sx, T, grad[w][off[i]:off[i + 1]].view(m, k),
                                  workspace=ws)
        gq.gq_mx4_quantize(grad, sg, qg)
        gq.gq_mx4_reduce_dequant(qg, sg, 1, n, total)
        gq.gq_ortho_step(plan, total, update, in_mul=1.0 / W, momentum=momentum, mu=0.9)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    coded = []
    for w in range(W):
        g = grad[w].cpu().numpy()
        for i, (m, k) in enumerate(shapes):
            a = ref.decode(*ref.quantize(acts[w][i][0].float().cpu().numpy().T), T)
            b = ref.decode(*ref.quantize(acts[w][i][1].float().cpu().numpy().T), T)
            # T sums, each within a unit of the last place of the sum of |a b|
            d = np.abs(g[off[i]:off[i + 1]].reshape(m, k) - a @ b.T)
            assert np.all(d <= (T + 2) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T))
        coded.append(ref.quantize(g.reshape(1, -1)))
    want = ref.reduce([c[0] for c in coded], [c[1] for c in coded], n).reshape(-1)
    assert np.array_equal(total.cpu().numpy(), want)
    g = want * np.float32(1.0 / W)
    u = (g + np.float32(0.9) * g).astype(np.float64)
    for i, (m, k) in enumerate(shapes):
        x, bound = iterate(u[off[i]:off[i + 1]].reshape(m, k), [COEF] * 5)
        _check(update[off[i]:off[i + 1]].double().cpu().numpy().reshape(m, k), x, bound, "bf16")
    first = [t.clone() for t in (total, update, momentum)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for run in (graph.replay, step):
            for t in (total, update, momentum):
                t.zero_()
            run()
            torch.cuda.synchronize()
            for t, f in zip((total, update, momentum), first):
                assert torch.equal(t, f), i


def test_readme_programs_run(gq):
    text = (pathlib.Path(__file__).resolve().parent.parent / "README.md").read_text()
    names = {}
    programs = re.findall(r"```python\n(.*?)```", text, re.S)
    assert len(programs) == 2
    for p in programs:
        exec(p, names)
    torch.cuda.synchronize()
    update = names["update"].float()
    # an orthogonalised matrix: the default coefficients leave singular values
    # between 0.68 and 1.13 of directions that are not lost, and 1024 of them
    assert bool(torch.isfinite(update).all()) and 0 < float(update.norm()) <= 1.2 * 32
