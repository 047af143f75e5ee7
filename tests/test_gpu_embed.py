"""gq_embed and gq_embed_grad on the GPU against their definitions.

Tolerances.  A lookup is exact by definition (one product rounded to binary32,
then to the output's type) and is compared bit for bit.  A gradient row is a
sum of k terms in binary32, in an order of the library's choice: off by at most
(k - 1) 2^-24 (1 + k 2^-24) sum |dy|; the product with mul adds 2^-24 of the
result, the accumulation 2^-24 of what it gives, and the output's type half a
step (2^-24, 2^-11, 2^-8 relative, and half of its smallest subnormal).  Sums
of small whole numbers are exact in any order and compared bit for bit."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": (2.0 ** -24, 2.0 ** -150), "f16": (2.0 ** -11, 2.0 ** -25),
        "bf16": (2.0 ** -8, 2.0 ** -134)}
GUARD = -77.0


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _wide(rows, cols, gap, dt, shift=0):
    """(rows x cols view, its whole buffer) of rows `gap` elements apart, from
    element `shift` of the buffer on; filled with a guard value."""
    flat = torch.full((rows * (cols + gap) + shift + 8,), GUARD, dtype=TORCH[dt], device="cuda")
    return flat[shift:shift + rows * (cols + gap)].view(rows, cols + gap)[:, :cols], flat


def _untouched(view, flat):
    """That nothing of the buffer but the view was written."""
    view.fill_(GUARD)
    assert bool((flat == GUARD).all()), "wrote outside the rows"


def _bits(a, b):
    v = {4: torch.int32, 2: torch.int16}[a.element_size()]
    nan = torch.isnan(a) & torch.isnan(b)
    return bool(((a.contiguous().view(v) == b.contiguous().view(v)) | nan).all())


def _idx(rng, T, V, kind, it):
    """Indexes: evenly spread, skewed, all alike, every row in turn, with some
    outside the table."""
    if kind == "even":
        i = rng.integers(0, V, T)
    elif kind == "skewed":
        i = np.minimum((V + 1) ** rng.random(T) - 1, V - 1).astype(np.int64)
        i = rng.permutation(V)[i]
    elif kind == "one":
        i = np.full(T, V // 2)
    elif kind == "turn":
        i = np.arange(T) % V
    else:
        i = rng.integers(-3, V + 3, T)
        big = 2 ** 31 - 1 if it == torch.int32 else 2 ** 62
        i[rng.random(T) < 0.1] = big
        i[rng.random(T) < 0.1] = -big
    return torch.from_numpy(np.asarray(i, np.int64)).to(it).cuda()


def _lookup(idx, table, mul, dt):
    i = idx.long().view(-1)
    ok = (i >= 0) & (i < table.shape[0])
    x = table[i.clamp(0, table.shape[0] - 1)].float() * torch.tensor(mul, device="cuda")
    return torch.where(ok[:, None], x, torch.zeros((), device="cuda")).to(dt)


SIZES = [(1, 1, 1), (1, 5, 16), (2, 3, 7), (5, 2, 64), (3, 100, 1000), (257, 50, 129),
         (1000, 300, 33), (64, 7, 4100), (513, 1000, 8), (4097, 33, 5)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_lookup(gq, dt, out):
    rng = np.random.default_rng(1)
    for k, (T, V, D) in enumerate(SIZES):
        for kind in ("even", "one", "outside"):
            it = (torch.int32, torch.int64)[k % 2]
            gap, shift, mul = (0, 1, 3)[k % 3], k % 4, (1.0, 0.37, -32.0)[k % 3]
            say("lookup", dt, out, T, V, D, kind, "gap", gap, "shift", shift)
            table, _ = _wide(V, D, gap, dt, shift)
            table.copy_(torch.from_numpy(rng.standard_normal((V, D)).astype(np.float32)))
            if V > 2 and D > 2:
                table[1, 1], table[1, 2], table[0, 0] = float("inf"), float("nan"), -0.0
            idx = _idx(rng, T, V, kind, it)
            o, flat = _wide(T, D, gap, out, shift)
            gq.gq_embed(idx, table, o, mul=mul)
            assert _bits(o, _lookup(idx, table, mul, TORCH[out])), (T, V, D, kind)
            _untouched(o, flat)


@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16"),
                                    ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,D", [(9001, 1024), (9001, 1029), (140_003, 40), (530_003, 5),
                                 (5000, 4100), (40_000, 129)])
def test_long_lookup(gq, dt, out, T, D):
    """Lookups of several slabs a wave, with the output's rows on every offset
    from a line of memory."""
    rng = np.random.default_rng(T + D)
    V = 97
    table, _ = _wide(V, D, 0, dt)
    table.copy_(torch.from_numpy(rng.standard_normal((V, D)).astype(np.float32)))
    for gap, shift in ((0, 0), (0, 1), (3, 2), (64, 32)):
        say("long lookup", dt, out, T, D, "gap", gap, "shift", shift)
        idx = _idx(rng, T, V, "outside", torch.int32 if gap else torch.int64)
        o, flat = _wide(T, D, gap, out, shift)
        gq.gq_embed(idx, table, o, mul=0.37)
        assert _bits(o, _lookup(idx, table, 0.37, TORCH[out])), (gap, shift)
        _untouched(o, flat)


def _sum64(idx, dy, V, mul, skip):
    """(the gradient, sum of magnitudes, tokens of each row) in 64 bits."""
    i = idx.long().view(-1).cpu()
    ok = (i >= 0) & (i < V) & (i != (-1 if skip is None else skip))
    x = dy.double().cpu()[ok]
    g, m = torch.zeros(V, x.shape[1], dtype=torch.float64), torch.zeros(V, x.shape[1],
                                                                        dtype=torch.float64)
    g.index_add_(0, i[ok], x)
    m.index_add_(0, i[ok], x.abs())
    mul = float(np.float32(mul))
    return g * mul, m * abs(mul), torch.bincount(i[ok], minlength=V).double()


def _check(got, base, idx, dy, V, mul, skip, out, what):
    g, m, k = _sum64(idx, dy, V, mul, skip)
    half, least = HALF[out]
    k = k[:, None]
    err = (k - 1).clamp(min=0) * 2.0 ** -24 * (1 + k * 2.0 ** -24) * m
    err = err + (g.abs() + err) * 2.0 ** -24 + 2.0 ** -149
    if base is not None:
        g = g + base.double().cpu()
    err = err + (g.abs() + err) * half + least
    off = (got.double().cpu() - g).abs()
    assert bool((off <= err).all()), (what, float((off - err).max()), float((off / err).max()))
    empty = (k == 0).expand_as(g)
    if base is None:
        assert bool((got.cpu()[empty] == 0).all()), (what, "rows without a token")
    else:
        assert bool((got.cpu()[empty] == base.cpu()[empty]).all()), (what, "rows without a token")


def _grad(gq, idx, dy, grad, **kw):
    n = gq.gq_embed_grad_workspace(idx.numel(), *grad.shape)
    ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    gq.gq_embed_grad(idx, dy, grad, ws[:n], **kw)
    assert bool((ws[n:] == 0xA5).all()), "wrote past the workspace"


# gradients of more tokens than one launch takes, of few and many columns
LONG = [(3000, 1, 20), (20_000, 4, 9), (9000, 30_522, 24), (2049, 300, 16), (2500, 40, 17),
        (3000, 90, 64), (3000, 90, 65), (5000, 20, 128), (5000, 2000, 129), (2100, 33, 1030),
        (1200, 90, 2000), (40, 12, 60_000)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16", "add"])
def test_gradient(gq, dt, out):
    rng = np.random.default_rng(2)
    add, out = out == "add", "f32" if out == "add" else out
    for k, (T, V, D) in enumerate(SIZES + LONG):
        for j, kind in enumerate(("even", "skewed", "one", "outside")):
            it = (torch.int32, torch.int64)[(k + j) % 2]
            gap, shift, mul = (0, 1, 3)[(k + j) % 3], k % 4, (1.0, 0.37, -32.0)[k % 3]
            skip = (None, V // 2, 0, V + 1)[(k + j) % 4]
            say("gradient", dt, out, "add" if add else "", T, V, D, kind, "skip", skip, "gap", gap)
            idx = _idx(rng, T, V, kind, it)
            dy, _ = _wide(T, D, gap, dt, shift)
            dy.copy_(torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)))
            grad, flat = _wide(V, D, gap, out, shift)
            base = None
            if add:
                base = torch.from_numpy(rng.standard_normal((V, D)).astype(np.float32)).cuda()
                grad.copy_(base)
            _grad(gq, idx, dy, grad, mul=mul, skip=skip, accumulate=add)
            _check(grad, base, idx, dy, V, mul, skip, out, (T, V, D, kind))
            _untouched(grad, flat)


@pytest.mark.parametrize("V", [1, 2, 63, 255, 256, 257, 1000, 30_522, 262_144, 262_145, 700_001])
def test_whole_numbers(gq, V):
    """Sums of small whole numbers, exact in any order: every row count the
    sort's ranges can have, and runs of every length."""
    rng = np.random.default_rng(V)
    for T in (0, 1, 63, 64, 65, 1000, 16_384, 70_001):
        for kind in ("even", "skewed", "turn", "outside"):
            say("whole numbers", V, T, kind)
            idx = _idx(rng, T, V, kind, torch.int64)
            dy = torch.from_numpy(rng.integers(-4, 5, (T, 3)).astype(np.float32)).cuda()
            grad = torch.full((V, 3), GUARD, device="cuda")
            _grad(gq, idx, dy, grad)
            i = idx.cpu()
            ok = (i >= 0) & (i < V)
            want = torch.zeros(V, 3, dtype=torch.float64).index_add_(0, i[ok], dy.cpu()[ok].double())
            assert bool((grad.cpu().double() == want).all()), (V, T, kind)


@pytest.mark.parametrize("D", [1, 16, 31, 64, 100, 512, 1025])
def test_runs_of_every_length(gq, D):
    """Row r has r tokens, scattered over the batch; long and short runs
    meet at every offset."""
    rng = np.random.default_rng(D)
    runs = np.concatenate([np.arange(0, 140), [200, 255, 256, 257, 300, 511, 512, 513, 1025, 2000]])
    i = rng.permutation(np.repeat(np.arange(runs.size), runs))
    idx = torch.from_numpy(i).cuda()
    dy = torch.from_numpy(rng.integers(-4, 5, (i.size, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    grad = torch.full((runs.size, D), GUARD, device="cuda")
    _grad(gq, idx, dy, grad)
    want = torch.zeros(runs.size, D, dtype=torch.float64).index_add_(0, idx.cpu(), dy.cpu().double())
    assert bool((grad.cpu().double() == want).all())


def test_difference(gq):
    """The gradient of sum(w * lookup(table)) against its differences: the
    lookup is linear, and with powers of two both are exact."""
    rng = np.random.default_rng(4)
    V, D, T, mul = 11, 6, 40, 0.5
    table = torch.from_numpy(rng.integers(-8, 9, (V, D)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.integers(-8, 9, (T, D)).astype(np.float32)).cuda()
    idx = _idx(rng, T, V, "outside", torch.int64)
    grad = torch.empty(V, D, device="cuda")
    _grad(gq, idx, w, grad, mul=mul)

    def loss(t):
        o = torch.empty(T, D, device="cuda")
        gq.gq_embed(idx, t, o, mul=mul)
        return float((o.double() * w.double()).sum())

    for r in range(V):
        for c in range(D):
            up, down = table.clone(), table.clone()
            up[r, c] += 1.0
            down[r, c] -= 1.0
            assert (loss(up) - loss(down)) / 2 == float(grad[r, c]), (r, c)


def test_non_finite(gq):
    """inf and NaN stay in the rows whose tokens hold them; those of left-out
    tokens reach nothing."""
    idx = torch.tensor([0, 1, 2, 3, -1, 9, 2, 4], device="cuda")
    dy = torch.ones(8, 70, device="cuda")
    dy[1, 3], dy[2, 5], dy[6, 5] = float("nan"), float("inf"), float("-inf")
    dy[4], dy[5], dy[7] = float("nan"), float("inf"), float("nan")
    grad = torch.empty(5, 70, device="cuda")
    _grad(gq, idx, dy, grad, skip=4)
    want = torch.ones(5, 70)
    want[1, 3], want[2], want[4] = float("nan"), 2.0, 0.0
    want[2, 5] = float("nan")
    assert _bits(grad.cpu(), want)


def test_repeats_streams_and_no_tokens(gq):
    rng = np.random.default_rng(5)
    T, V, D = 5000, 900, 200
    idx = _idx(rng, T, V, "skewed", torch.int64)
    dy = torch.randn(T, D, device="cuda")
    n = gq.gq_embed_grad_workspace(T, V, D)
    want = torch.empty(V, D, device="cuda")
    _grad(gq, idx, dy, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in streams]
    got = [torch.empty(20, V, D, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, w, g in zip(streams, ws, got):
            with torch.cuda.stream(s):
                gq.gq_embed_grad(idx, dy, g[i], w)
    torch.cuda.synchronize()
    for g in got:
        assert all(_bits(x, want) for x in g)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    g = torch.full((V, D), GUARD, device="cuda")
    _grad(gq, none, torch.empty(0, D, device="cuda"), g, accumulate=True)
    assert bool((g == GUARD).all())
    _grad(gq, none, torch.empty(0, D, device="cuda"), g)
    assert bool((g == 0).all())
    gq.gq_embed(none, g, torch.empty(0, D, device="cuda"))
    torch.cuda.synchronize()


def test_captured(gq):
    """Lookup and gradient in one graph, replayed on new tokens, with eager
    calls on the same workspace between the replays."""
    rng = np.random.default_rng(6)
    T, V, D = 3000, 500, 96
    idx = torch.zeros(T, dtype=torch.int64, device="cuda")
    table = torch.randn(V, D, device="cuda")
    o = torch.empty(T, D, device="cuda", dtype=torch.bfloat16)
    grad, eager = torch.zeros(V, D, device="cuda"), torch.zeros(V, D, device="cuda")
    ws = torch.empty(gq.gq_embed_grad_workspace(T, V, D), dtype=torch.uint8, device="cuda")
    gq.gq_embed(idx, table, o)
    gq.gq_embed_grad(idx, o, grad, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gq.gq_embed(idx, table, o, mul=2.0)
        gq.gq_embed_grad(idx, o, grad, ws, skip=3)
    for k in range(5):
        idx.copy_(_idx(rng, T, V, ("skewed", "one", "outside", "even", "turn")[k], torch.int64))
        table.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert _bits(o, _lookup(idx, table, 2.0, torch.bfloat16)), k
        gq.gq_embed_grad(idx, o, eager, ws, skip=3)
        torch.cuda.synchronize()
        assert _bits(grad, eager), k
        _check(grad, None, idx, o, V, 1.0, 3, "f32", k)


def test_above_2_32_elements(gq):
    """Tables, outputs and gradients whose offsets pass 32 bits."""
    V, D = (1 << 22) + 3, 1028
    table = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, (1 << 21) - 1, 1 << 22, V - 1]
    for r in rows:
        table[r] = r % 97 + 1
    idx = torch.tensor(rows + [7], device="cuda")
    o = torch.empty(6, D, dtype=torch.bfloat16, device="cuda")
    gq.gq_embed(idx, table, o)
    assert [float(v) for v in o[:, D - 1]] == [r % 97 + 1 for r in rows] + [0]
    del o
    dy = torch.ones(6, D, dtype=torch.bfloat16, device="cuda") * torch.arange(
        1, 7, device="cuda")[:, None]
    idx[5] = rows[4]
    _grad(gq, idx, dy, table)
    got = torch.nonzero(table[:, D - 1]).view(-1).tolist()
    assert got == sorted(rows)
    assert [float(table[r, 0]) for r in rows] == [1, 2, 3, 4, 11]
    assert float(table.sum(dtype=torch.float32)) == 21.0 * D
    # as many tokens
    T = (1 << 22) + 5
    idx = torch.zeros(T, dtype=torch.int32, device="cuda")
    idx[T - 1] = 1
    o = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    small = torch.tensor([1.0, 2.0], device="cuda")[:, None].expand(2, D).contiguous()
    gq.gq_embed(idx, small, o)
    assert float(o[T - 1, D - 1]) == 2 and float(o[T - 2, 0]) == 1
    grad = torch.empty(2, D, device="cuda")
    o.zero_()
    o[T - 1], o[T - 2], o[5] = 3.0, 5.0, 7.0
    _grad(gq, idx, o, grad)
    assert bool((grad[0] == 12).all()) and bool((grad[1] == 3).all())


@pytest.mark.parametrize("more", [150, 3000])
def test_most_rows(gq, more):
    """The largest number of rows, with a token in the first, the last and two
    between, and `more` of one row."""
    V = 1 << 30
    grad = torch.full((V, 1), GUARD, dtype=torch.float16, device="cuda")
    idx = torch.tensor([V - 1, 0, V // 3, V // 2 + 1, V, -1] + [V - 2] * more, device="cuda")
    dy = torch.ones(idx.numel(), 1, dtype=torch.float16, device="cuda")
    dy[:6, 0] = torch.arange(1, 7)
    dy[150:, 0] = 0                         # (sums up to 2048 are whole numbers of fp16)
    _grad(gq, idx, dy, grad)
    at = [V - 1, 0, V // 3, V // 2 + 1, V - 2]
    assert [float(grad[i, 0]) for i in at] == [1, 2, 3, 4, 144]
    assert int((grad != 0).sum()) == 5


@pytest.mark.parametrize("T", [3, 2049])
def test_most_columns(gq, T):
    """The largest number of columns, of few tokens and of pieces whose slabs fill
    more than one side of a grid."""
    D, V = 1 << 24, 2
    idx = torch.zeros(T, dtype=torch.int32, device="cuda")
    idx[1] = 1
    dy = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    places = [0, 511, 512, D // 2 + 3, D - 1]
    for p in places:
        dy[:, p] = 1.0
    grad = torch.full((V, D), GUARD, device="cuda")
    _grad(gq, idx, dy, grad)
    assert [float(grad[0, p]) for p in places] == [T - 1] * 5
    assert [float(grad[1, p]) for p in places] == [1] * 5
    assert float(grad.double().sum()) == 5 * T
    out = torch.full((T, D), GUARD, dtype=torch.bfloat16, device="cuda") if T == 3 else dy
    gq.gq_embed(idx, grad, out, mul=0.5)
    assert [float(out[1, p]) for p in places] == [0.5] * 5 and float(out[1].double().sum()) == 2.5
    assert [float(out[T - 1, p]) for p in places] == [0.5 * (T - 1)] * 5


def test_single_vectors(gq):
    """One token's output and gradient as vectors, the form of decoding."""
    table = torch.randn(9, 70, device="cuda")
    idx = torch.tensor([4], dtype=torch.int32, device="cuda")
    o = torch.empty(70, device="cuda")
    gq.gq_embed(idx, table, o)
    assert torch.equal(o, table[4])
    grad = torch.full((9, 70), GUARD, device="cuda")
    _grad(gq, idx, o, grad)
    assert torch.equal(grad[4], o) and int((grad != 0).any(1).sum()) == 1


def test_most_tokens(gq):
    """More tokens than a wave's list can number: 2^26 and some, of whole
    numbers."""
    T, V = (1 << 26) + 5003, 70_001
    gen = torch.Generator(device="cuda").manual_seed(7)
    idx = torch.randint(-1, V, (T,), dtype=torch.int32, device="cuda", generator=gen)
    dy = torch.randint(-4, 5, (T, 1), device="cuda", generator=gen).to(torch.bfloat16)
    grad = torch.full((V, 1), GUARD, device="cuda")
    _grad(gq, idx, dy, grad, skip=5)
    i = torch.where((idx >= 0) & (idx != 5), idx, torch.full_like(idx, V)).long()
    want = torch.zeros(V + 1, dtype=torch.float64, device="cuda").index_add_(0, i, dy[:, 0].double())
    assert bool((grad[:, 0].double() == want[:V]).all())


# gradients whose rows without a token are cleared by work groups of their own, among
# those of the sums: four rows or more a token, of 1 KiB or more
MANY_ROWS = [(2049, 8196, 256), (2100, 8403, 257), (2100, 8403, 513), (2500, 10_007, 1030),
             (300, 8192, 14_003), (16_500, 66_007, 512)]


@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16"),
                                    ("bf16", "bf16")])
def test_rows_cleared_beside_the_sums(gq, dt, out):
    """Sums of small whole numbers, exact in any order, in a gradient of which
    every element has to be written, and nothing else."""
    rng = np.random.default_rng(9)
    for k, (T, V, D) in enumerate(MANY_ROWS):
        for j, kind in enumerate(("even", "skewed", "one", "outside", "first", "last")):
            it = (torch.int32, torch.int64)[(k + j) % 2]
            gap, shift, skip = (0, 1, 3)[(k + j) % 3], (k + j) % 4, (None, 0, V // 2)[j % 3]
            say("cleared beside the sums", dt, out, T, V, D, kind, "skip", skip, "gap", gap)
            if kind == "first":
                idx = torch.arange(T, dtype=it, device="cuda")
            elif kind == "last":
                idx = torch.arange(V - T, V, dtype=it, device="cuda").flip(0)
            else:
                idx = _idx(rng, T, V, kind, it)
            dy, _ = _wide(T, D, gap, dt, shift)
            dy.copy_(torch.from_numpy(rng.integers(-4, 5, (T, D)).astype(np.float32)))
            grad, flat = _wide(V, D, gap, out, shift)
            _grad(gq, idx, dy, grad, skip=skip)
            i = idx.long()
            ok = (i >= 0) & (i < V) & (i != (-1 if skip is None else skip))
            want = torch.zeros(V, D, dtype=torch.float64, device="cuda")
            want.index_add_(0, i[ok], dy.double()[ok])
            # (one rounding of a whole number below 2^24; zeros are +0)
            assert _bits(grad, (want + 0.0).to(TORCH[out])), (T, V, D, kind)
            _untouched(grad, flat)
            del dy, grad, flat, want
