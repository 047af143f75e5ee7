"""The microscaled 4-bit exchange and product on the GPU against the plain
numpy implementation (tests/mx4_ref.py).  Codes, scales and rank-order sums
are exact by definition and compared bit for bit; the product's tolerance is
the rounding bound of its binary32 sums."""
import numpy as np
import pytest
import torch

from tests import mx4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GUARD = 64


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _values(rng, rows, cols, dt):
    """Gradients of every binade, zeros of both signs, subnormals, values half
    way between codes, blocks of zeros, and a few inf and NaN."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 3, (rows, 1)))
    ties = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 0., -0., 4])
    pick = rng.random((rows, cols))
    x = np.where(pick < 0.3, rng.choice(ties, (rows, cols)) * rng.choice([-1, 1], (rows, cols)), x)
    big = 2.0 ** 100 if dt != "f16" else 2.0 ** 10
    nb = ref.blocks(cols)
    for b in range(nb):
        kind = rng.integers(0, 12)
        r = rng.integers(0, rows)
        c = slice(32 * b, min(cols, 32 * b + 32))
        if kind == 0:
            x[r, c] = rng.choice([0., -0.])
        elif kind == 1:
            x[r, c] *= 2.0 ** -149 if dt != "f16" else 2.0 ** -24
        elif kind == 2:
            x[r, c] *= big
        elif kind == 3:
            x[r, rng.integers(32 * b, c.stop)] = rng.choice([np.inf, -np.inf, np.nan])
    with np.errstate(over="ignore"):
        return torch.from_numpy(x.astype(np.float32)).to(TORCH[dt])


def _same(got, want, what):
    got = got.cpu().numpy().reshape(-1)
    want = np.asarray(want).reshape(-1)
    bad = np.flatnonzero(got != want)
    assert bad.size == 0, (what, int(bad[0]), int(got[bad[0]]), int(want[bad[0]]), bad.size)


def _same_f32(got, want, what):
    g = got.cpu().numpy().reshape(-1)
    w = np.asarray(want, np.float32).reshape(-1)
    bad = np.flatnonzero((g.view(np.uint32) != w.view(np.uint32)) & ~(np.isnan(g) & np.isnan(w)))
    assert bad.size == 0, (what, int(bad[0]), g[bad[0]], w[bad[0]], bad.size)


def _out(n):
    return torch.full((n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")


def _guards(*ts):
    for t in ts:
        assert bool((t[-GUARD:] == 0xA5).all()), "wrote past the end"


SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (1, 4097), (1, 20000), (3, 5), (5, 64), (7, 100),
          (33, 32), (64, 1), (130, 257), (31, 1024), (2, 33000)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize(gq, dt, transpose):
    rng = np.random.default_rng(3)
    for rows, cols in SHAPES:
        for W, mul, gap in ((1, 1.0, 0), (3, 2.0 ** -16, 0), (2, 0.3, 8), (1, 1.0, 3)):
            say("quantize", dt, transpose, rows, cols, "W", W, "mul", mul, "gap", gap)
            xs = []
            for w in range(W):
                wide = torch.zeros(rows, cols + gap, dtype=TORCH[dt])
                wide[:, :cols] = _values(rng, rows, cols, dt)
                xs.append(wide.cuda()[:, :cols])
            n, b = gq.gq_mx4_sizes(*((cols, rows) if transpose else (rows, cols)))
            sc, q = [_out(n) for _ in range(W)], [_out(b) for _ in range(W)]
            gq.gq_mx4_quantize(xs, sc, q, in_mul=mul, transpose=transpose)
            for w in range(W):
                x = xs[w].float().cpu().numpy()
                s_ref, q_ref = ref.quantize(x.T if transpose else x, mul)
                _same(sc[w][:n], s_ref, "scale")
                _same(q[w][:b], q_ref, "codes")
                _guards(sc[w], q[w])


def _random_codes(rng, rows, cols, lo=100, hi=140, nan=0.0):
    nb = ref.blocks(cols)
    c = rng.integers(0, 16, (rows, nb * 32)).astype(np.uint8)
    c[:, cols:] = 0
    q = (c[:, 0::2] | c[:, 1::2] << 4).reshape(rows, nb, 16)
    s = rng.integers(lo, hi, (rows, nb)).astype(np.uint8)
    s[rng.random((rows, nb)) < nan] = 255
    return s, q


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).reshape(-1)).cuda()


@pytest.mark.parametrize("W", [1, 2, 7, 8, 9, 64])
def test_reduce(gq, W):
    rng = np.random.default_rng(W)
    for rows, cols in SHAPES:
        for lo, hi, nan in ((100, 140, 0.02), (0, 40, 0.0), (0, 253, 0.0)):
            say("reduce W", W, rows, cols, lo, hi)
            ranks = [_random_codes(rng, rows, cols, lo, hi, nan) for _ in range(W)]
            with np.errstate(over="ignore"):
                r = ref.reduce([s for s, _ in ranks], [q for _, q in ranks], cols)
            sc, q = [_dev(s) for s, _ in ranks], [_dev(c) for _, c in ranks]
            n, b = gq.gq_mx4_sizes(rows, cols)
            out = torch.full((rows * cols + GUARD,), -7.0, device="cuda")
            gq.gq_mx4_reduce_dequant(q, sc, rows, cols, out)
            _same_f32(out[:rows * cols], r, "sum")
            assert bool((out[rows * cols:] == -7).all())
            s_ref, q_ref = ref.quantize(r)
            for with_r in (False, True):
                so, qo = _out(n), _out(b)
                out.fill_(-7.0)
                gq.gq_mx4_reduce_requantize(q, sc, rows, cols, so, qo, r_out=out if with_r else None)
                _same(so[:n], s_ref, "scale")
                _same(qo[:b], q_ref, "codes")
                _guards(so, qo)
                if with_r:
                    _same_f32(out[:rows * cols], r, "fused sum")
                assert bool((out[rows * cols:] == -7).all())


PRODUCTS = [(1, 1, 1), (1, 1, 33), (3, 5, 31), (16, 16, 128), (17, 33, 100), (64, 64, 256),
            (65, 63, 257), (7, 1000, 1024), (128, 130, 513), (300, 200, 4096), (64, 147, 4000),
            (1, 30, 4096), (1000, 24, 2000), (513, 511, 640), (1100, 4200, 300), (70, 60, 2600),
            (4000, 4097, 520), (2049, 2050, 33)]


def _product(gq, rng, m, n, k, dt, add, split, gap, offset, lo, hi, nan=0.0):
    sa, qa = _random_codes(rng, m, k, lo, hi, nan)
    sb, qb = _random_codes(rng, n, k, lo, hi, nan)
    c0 = rng.standard_normal((m, n)).astype(np.float32)
    flat = torch.full((offset + m * (n + gap) + GUARD,), -7.0, dtype=TORCH[dt], device="cuda")
    c = flat[offset:offset + m * (n + gap)].view(m, n + gap)[:, :n]
    if add:
        c.copy_(torch.from_numpy(c0))
    before = flat.clone()
    ws = None
    if split:
        ws = torch.full((gq.gq_mx4_product_workspace(m, n, k) + 16,), 0xA5, dtype=torch.uint8,
                        device="cuda")
    gq.gq_mx4_product(_dev(qa), _dev(sa), _dev(qb), _dev(sb), k, c, accumulate=add, workspace=ws)
    got = c.double().cpu().numpy()
    c.copy_(before[offset:offset + m * (n + gap)].view(m, n + gap)[:, :n])
    assert torch.equal(flat, before), "wrote outside the matrix"
    a, b = ref.decode(sa, qa, k), ref.decode(sb, qb, k)
    return got, a, b, c0.astype(np.float64)


def test_product_of_small_integers_is_exact(gq):
    """Scales 126 .. 128: every term is a multiple of 2^-4 and k <= 4096
    terms stay below 4096 * 36 * 4 < 2^20, so binary32 sums are exact in any
    order and every bit is fixed."""
    rng = np.random.default_rng(5)
    for m, n, k in PRODUCTS:
        for split in (False, True):
            say("exact product", m, n, k, "split", split)
            got, a, b, _ = _product(gq, rng, m, n, k, "f32", False, split, 0, 0, 126, 129)
            bad = np.argwhere(got != a @ b.T)
            assert bad.size == 0, (m, n, k, split, bad[0], len(bad))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_product(gq, dt):
    """|c - exact| <= (k + 2) * 2^-23 * sum|a b| (k sums and the join, each
    within one unit, two half steps), plus half a step of c's type."""
    rng = np.random.default_rng(7)
    half = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dt]
    least = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}[dt]
    for m, n, k in PRODUCTS:
        for add, split, gap, offset in ((False, True, 0, 0), (dt == "f32", False, 5, 1),
                                        (dt == "f32", True, 4, 3)):
            say("product", dt, m, n, k, "add", add, "split", split, "gap", gap, "offset", offset)
            got, a, b, c0 = _product(gq, rng, m, n, k, dt, add, split, gap, offset, 120, 128)
            want = a @ b.T + (c0 if add else 0.0)
            size = np.abs(a) @ np.abs(b).T + (np.abs(c0) if add else 0.0)
            tol = (k + 2) * 2.0 ** -23 * size + half * np.abs(want) * (1 + 2.0 ** -8) + least
            assert np.all(np.abs(got - want) <= tol), (m, n, k, np.abs(got - want).max())


def test_product_nan_scale(gq):
    rng = np.random.default_rng(8)
    for m, n, k in ((40, 50, 200), (300, 290, 96)):
        say("nan", m, n, k)
        sa, qa = _random_codes(rng, m, k, 120, 130)
        sb, qb = _random_codes(rng, n, k, 120, 130)
        sa[3, 1] = 255
        sb[7, 2] = 255
        c = torch.zeros(m, n, device="cuda")
        gq.gq_mx4_product(_dev(qa), _dev(sa), _dev(qb), _dev(sb), k, c)
        nan = torch.isnan(c).cpu().numpy()
        want = np.zeros((m, n), bool)
        want[3, :] = True
        want[:, 7] = True
        assert np.array_equal(nan, want)


def test_product_repeats_bit_for_bit(gq):
    rng = np.random.default_rng(9)
    m, n, k = 130, 140, 9000
    sa, qa = _random_codes(rng, m, k, 100, 140)
    sb, qb = _random_codes(rng, n, k, 100, 140)
    args = [_dev(v) for v in (qa, sa, qb, sb)]
    ws = torch.empty(gq.gq_mx4_product_workspace(m, n, k), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    first = None
    for _ in range(5):
        c = torch.empty(m, n, device="cuda")
        ws.fill_(0xFF)
        gq.gq_mx4_product(*args, k, c, workspace=ws)
        first = c if first is None else first
        assert torch.equal(c, first)


def test_weight_gradient_exchange_run(gq):
    """The operators as a training step uses them: two ranks' weight
    gradients from 4-bit activations, added over two micro-batches into the
    flat fp32 gradient, exchanged in 4 bits, all on a stream of their own and
    then captured and replayed."""
    rng = np.random.default_rng(10)
    T, m, n, W = 96, 40, 52, 2
    dy = [[torch.from_numpy(rng.standard_normal((T, m)).astype(np.float32)).bfloat16().cuda()
           for _ in range(2)] for _ in range(W)]
    x = [[torch.from_numpy(rng.standard_normal((T, n)).astype(np.float32)).bfloat16().cuda()
          for _ in range(2)] for _ in range(W)]

    def buf(k):
        return torch.empty(k, dtype=torch.uint8, device="cuda")

    ny, by = gq.gq_mx4_sizes(m, T)
    nx, bx = gq.gq_mx4_sizes(n, T)
    ng, bg = gq.gq_mx4_sizes(1, m * n)
    sy, qy, sx, qx = buf(ny), buf(by), buf(nx), buf(bx)
    grad = [torch.zeros(m * n, device="cuda") for _ in range(W)]
    sg, qg = [buf(ng) for _ in range(W)], [buf(bg) for _ in range(W)]
    so, qo, r = buf(ng), buf(bg), torch.empty(m * n, device="cuda")

    def step():
        for w in range(W):
            grad[w].zero_()
            for mb in range(2):
                gq.gq_mx4_quantize([dy[w][mb]], [sy], [qy], transpose=True)
                gq.gq_mx4_quantize([x[w][mb]], [sx], [qx], transpose=True)
                gq.gq_mx4_product(qy, sy, qx, sx, T, grad[w].view(m, n), accumulate=True)
        gq.gq_mx4_quantize(grad, sg, qg)
        gq.gq_mx4_reduce_requantize(qg, sg, 1, m * n, so, qo, r_out=r)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    rs = []
    for w in range(W):
        g = np.zeros((m, n))
        for mb in range(2):
            a = ref.quantize(dy[w][mb].float().cpu().numpy().T)
            b = ref.quantize(x[w][mb].float().cpu().numpy().T)
            g += ref.decode(*a, T) @ ref.decode(*b, T).T
        # products of 4-bit values: sums of 192 of them are exact in binary32
        # up to the spread of the block scales; compared within its rounding
        got = grad[w].view(m, n).double().cpu().numpy()
        assert np.abs(got - g).max() <= (2 * T + 4) * 2.0 ** -23 * 36 * 2 * T
        rs.append(ref.quantize(grad[w].cpu().numpy().reshape(1, -1)))
        _same(sg[w], rs[w][0], "scale")
        _same(qg[w], rs[w][1], "codes")
    want = ref.reduce([v[0] for v in rs], [v[1] for v in rs], m * n)
    _same_f32(r, want, "sum")
    eager = [t.clone() for t in (r, so, qo)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        for t in (r, so, qo):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, e) for t, e in zip((r, so, qo), eager)), i
        step()
        torch.cuda.synchronize()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_short_rows_and_columns(gq, dt):
    """Every length around the pieces that the kernels load (1 to 17 elements
    and one more or less than 64 lanes), rows that start at any element, and
    1 to 9 blocks down the columns."""
    rng = np.random.default_rng(12)
    shapes = [(r, c) for r in (2, 9) for c in range(1, 18)] + [(3, 61), (3, 63), (2, 127)]
    shapes += [(r, c) for r in (31, 33, 64, 65, 97, 160, 257, 290) for c in (1, 2, 63, 65, 129, 300)]
    for rows, cols in shapes:
        for gap in (0, 1, 2):
            say("short", dt, rows, cols, "gap", gap)
            wide = torch.full((rows, cols + gap), float("nan"), dtype=TORCH[dt])
            wide[:, :cols] = _values(rng, rows, cols, dt)
            wide = wide.cuda()
            x = wide[:, :cols].float().cpu().numpy()
            for transpose in (False, True):
                s_ref, q_ref = ref.quantize(x.T if transpose else x)
                qr, qc = (cols, rows) if transpose else (rows, cols)
                n, b = gq.gq_mx4_sizes(qr, qc)
                sc, q = _out(n), _out(b)
                gq.gq_mx4_quantize([wide[:, :cols]], [sc], [q], transpose=transpose)
                _same(sc[:n], s_ref, "scale")
                _same(q[:b], q_ref, "codes")
                _guards(sc, q)
                out = torch.full((rows * cols + GUARD,), -7.0, device="cuda")
                gq.gq_mx4_reduce_dequant([q[:b]], [sc[:n]], qr, qc, out)
                _same_f32(out[:rows * cols], ref.reduce([s_ref], [q_ref], qc), "values")
                assert bool((out[rows * cols:] == -7).all())


def test_more_than_32_bits(gq):
    """Places above 2^32: elements of one long row, pieces of many short rows,
    and elements of the matrix that a product writes into.  The values are
    +-2^e and +-1.5 * 2^e, which a block of one element holds exactly, and,
    with e the same over a block, longer ones too."""
    def values(n):
        i = torch.arange(n, device="cuda", dtype=torch.int32)
        x = torch.where((i & 1) == 0, 1.0, 1.5).bfloat16()
        x *= torch.where((i & 64) == 0, 1.0, -1.0).bfloat16()
        x *= torch.where((i & 4096) == 0, 1.0, 2.0 ** -9).bfloat16()
        return x

    tile = values(1 << 20)
    n = (1 << 32) + 100
    x = tile.repeat(n // tile.numel() + 1)[:n]
    say("one row of", n)
    ns, nc = gq.gq_mx4_sizes(1, n)
    s, q = (torch.zeros(k, dtype=torch.uint8, device="cuda") for k in (ns, nc))
    r = torch.zeros(n, device="cuda")
    gq.gq_mx4_quantize([x], [s], [q])
    gq.gq_mx4_reduce_dequant([q], [s], 1, n, r)
    for lo in range(0, n, 1 << 30):
        assert torch.equal(r[lo:lo + (1 << 30)], x[lo:lo + (1 << 30)].float()), lo
    del x, s, q, r
    torch.cuda.empty_cache()
    rows = (1 << 30) + 77
    x = tile.repeat(rows // tile.numel() + 1)[:rows].view(rows, 1)
    say("rows of one", rows)
    ns, nc = gq.gq_mx4_sizes(rows, 1)
    s, q = (torch.zeros(k, dtype=torch.uint8, device="cuda") for k in (ns, nc))
    r = torch.zeros(rows, device="cuda")
    gq.gq_mx4_quantize([x], [s], [q])
    gq.gq_mx4_reduce_dequant([q], [s], rows, 1, r)
    assert torch.equal(r, x.view(-1).float())
    del x, s, q, r
    torch.cuda.empty_cache()
    m, k, ldc = 70, 300, 1 << 26
    say("product", m, m, k, "row stride", ldc)
    rng = np.random.default_rng(13)
    sa, qa = _random_codes(rng, m, k, 126, 129)
    a = ref.decode(sa, qa, k)
    big = torch.zeros(m * ldc, device="cuda")
    gq.gq_mx4_product(_dev(qa), _dev(sa), _dev(qa), _dev(sa), k, big.view(m, ldc)[:, :m])
    assert np.array_equal(big.view(m, ldc)[:, :m].double().cpu().numpy(), a @ a.T)
    big.view(m, ldc)[:, :m] = 0
    assert not bool(big.any())


def test_two_streams_at_once(gq):
    """Calls on two streams at once, which share their inputs and nothing
    else, and each with a workspace of its own."""
    rng = np.random.default_rng(14)
    m, n, k = 100, 90, 6000
    sa, qa = _random_codes(rng, m, k, 120, 130)
    sb, qb = _random_codes(rng, n, k, 120, 130)
    args = [_dev(v) for v in (qa, sa, qb, sb)]
    need = gq.gq_mx4_product_workspace(m, n, k)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in streams]
    c = [torch.zeros(m, n, device="cuda") for _ in streams]
    want = torch.zeros(m, n, device="cuda")
    gq.gq_mx4_product(*args, k, want, workspace=ws[0])
    torch.cuda.synchronize()
    for i in range(20):
        for j, st in enumerate(streams):
            gq.gq_mx4_product(*args, k, c[j], workspace=ws[j], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(c[0], want) and torch.equal(c[1], want)


def _exact_on_device(gq, m, n, k, split, seed):
    """Scales 126 and 127: terms are multiples of 2^-4 of at most 36, and for
    k <= 8192 their sums below 2^19, so every order of binary32 sums is exact,
    this product's and the library's (of the decoded values) alike."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nb = ref.blocks(k)

    def operand(rows):
        q = torch.randint(0, 256, (rows, nb * 16), dtype=torch.uint8, device="cuda", generator=gen)
        left = k - 32 * (nb - 1)            # elements of the last block
        last = q[:, (nb - 1) * 16:]
        last[:, (left + 1) // 2:] = 0
        if left % 2:
            last[:, left // 2] &= 15
        s = torch.randint(126, 128, (rows * nb,), dtype=torch.uint8, device="cuda", generator=gen)
        x = torch.empty(rows, k, device="cuda")
        gq.gq_mx4_reduce_dequant([q.reshape(-1)], [s], rows, k, x.view(-1))
        return q.reshape(-1), s, x

    qa, sa, a = operand(m)
    qb, sb, b = operand(n)
    c = torch.full((m, n), -7.0, device="cuda")
    ws = None
    if split:
        ws = torch.empty(gq.gq_mx4_product_workspace(m, n, k) + 16, dtype=torch.uint8, device="cuda")
    gq.gq_mx4_product(qa, sa, qb, sb, k, c, workspace=ws)
    assert torch.equal(c, torch.mm(a, b.t().contiguous())), (m, n, k, split)


def test_product_every_tile_and_length(gq):
    """Few and many tiles of each size, with K whole and in parts, and lengths
    around one, two, four and five groups of sixteen blocks."""
    for m, n in ((40, 50), (300, 200), (1000, 1100), (1030, 3000), (3499, 4095)):
        for k in (1, 100, 480, 511, 512, 530, 1100, 2047, 2048, 2049, 2100, 2600, 3500, 6200, 8192):
            for split in (False, True):
                say("exact on the device", m, n, k, "split", split)
                _exact_on_device(gq, m, n, k, split, m + k)


def test_product_nan_scale_of_every_tile(gq):
    """NaN scales in inner and in last rows and blocks reach their own row or
    column and nothing else, whatever lies behind the matrix."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    for m, n in ((40, 50), (1030, 3000), (3499, 4095)):
        for k in (96, 500, 530, 2049, 2600):
            say("nan", m, n, k)
            nb = ref.blocks(k)
            q = [torch.randint(0, 256, (r * nb * 16,), dtype=torch.uint8, device="cuda",
                               generator=gen) for r in (m, n)]
            s = [torch.full((r, nb), 127, dtype=torch.uint8, device="cuda") for r in (m, n)]
            rows, cols = [3, 17, m - 1], [7, 20, n - 1]
            for t, at in ((s[0], rows), (s[1], cols)):
                t[at[0], 1] = 255
                t[at[1], nb - 1] = 255
                t[at[2], nb - 1] = 255
            c = torch.zeros(m, n, device="cuda")
            gq.gq_mx4_product(q[0], s[0].view(-1), q[1], s[1].view(-1), k, c)
            want = torch.zeros(m, n, dtype=torch.bool, device="cuda")
            want[rows, :] = True
            want[:, cols] = True
            assert torch.equal(torch.isnan(c), want)
