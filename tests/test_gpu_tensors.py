"""gq_tensors_norm and gq_tensors_clip on the GPU against their definitions in
64 bits.

Tolerances.  A norm of n elements: each square is exact in binary64, and a sum
of n of them in any order is off by less than n 2^-53 relative; the root halves
that, the root itself, the product and in_mul's conversion add 3 2^-53; the one
rounding to binary32 is half a step, 2^-24 (2^-150 where the result is
subnormal).  The oracle's own sum is off by as much again.  A clip is exact by
definition (one rounding of f, of the product, and of the output type) and is
compared bit for bit."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TILE = 4096


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _norm64(xs, mul=1.0):
    return mul * np.sqrt(sum(float((x.double() ** 2).sum()) for x in xs))


def _near(got, want, n, what):
    got = float(got)
    bound = want * (2.0 ** -24 + (2 * n + 6) * 2.0 ** -53) + 2.0 ** -149
    assert abs(got - want) <= bound, (what, got, want, abs(got - want) / max(want, 1e-300))


def _make(lengths, dts, seed, scale=1.0, gap=0):
    """Tensors (on the device) of given lengths and types; with a gap, each a
    view into one buffer per type, `gap` elements behind the one before."""
    rng = torch.Generator().manual_seed(seed)
    xs = []
    flat = {d: torch.zeros(sum(m + gap for m, e in zip(lengths, dts) if e == d) + gap,
                           dtype=TORCH[d], device="cuda") for d in set(dts)}
    at = {d: gap for d in flat}
    for m, d in zip(lengths, dts):
        v = flat[d][at[d]:at[d] + m]
        v.copy_((torch.randn(m, generator=rng) * scale).to(TORCH[d]))
        at[d] += m + gap
        xs.append(v)
    return xs, flat


LENGTHS = [[1], [3], [64], [TILE], [TILE - 1], [TILE + 1], [1, 1, 1], [0, 5, 0], [0],
           [2 * TILE, 17, 3 * TILE + 5], [7, 100, 1000, 5000, 9], [250_001], [1] * 700,
           list(range(1, 300))]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16", "mixed"])
@pytest.mark.parametrize("gap", [0, 1, 3])
def test_norm(gq, dt, gap):
    for k, lengths in enumerate(LENGTHS):
        dts = [dt if dt != "mixed" else ("f32", "f16", "bf16")[i % 3] for i in range(len(lengths))]
        say("norm", dt, "gap", gap, "case", k, "tensors", len(lengths), "n", sum(lengths))
        xs, _ = _make(lengths, dts, 100 + k, gap=gap)
        t = gq.gq_tensors_create(xs)
        norm = torch.full((3,), 7.0, device="cuda")
        each = torch.full((len(xs) + 2,), 7.0, device="cuda")
        for mul in (1.0, 2.0 ** -16, 0.3):
            m = float(np.float32(mul))
            gq.gq_tensors_norm(t, norm, in_mul=mul)
            _near(norm[0], _norm64(xs, m), sum(lengths), (dt, gap, k, mul))
            gq.gq_tensors_norm(t, norm[1:], norms=each, in_mul=mul)
            _near(norm[1], _norm64(xs, m), sum(lengths), (dt, gap, k, mul, "with each"))
            for i, x in enumerate(xs):
                _near(each[i], _norm64([x], m), x.numel(), (dt, gap, k, mul, i))
        assert float(norm[2]) == 7.0 and bool((each[len(xs):] == 7.0).all()), "wrote past the end"
        assert gq.gq_tensors_info(t)["n"] == sum(lengths)


def test_norm_of_extreme_values(gq):
    """Squares that binary32 could not hold, and non-finite elements in every
    place of a tile."""
    norm, each = torch.empty(1, device="cuda"), torch.empty(3, device="cuda")
    for v in (1e-30, 2.0 ** -149, 1e30, 3e38):
        xs = [torch.full((n,), v, device="cuda") for n in (1, 5000, 33)]
        gq.gq_tensors_norm(gq.gq_tensors_create(xs), norm, norms=each)
        want = float(np.float32(v)) * np.sqrt(np.array([1, 5000, 33]))
        with np.errstate(over="ignore"):
            got = each.cpu().numpy()
            for g, w in zip(list(got) + [float(norm)], list(want) + [np.sqrt((want ** 2).sum())]):
                if w > 3.4028235e38 * (1 + 2.0 ** -24):
                    assert np.isinf(g)
                else:
                    assert abs(float(g) - w) <= w * (2.0 ** -24 + 2.0 ** -39) + 2.0 ** -149, (v, g, w)
    for dt in TORCH.values():
        for bad in (float("inf"), -float("inf"), float("nan")):
            for place in (0, 1, 4095, 4096, 5003, 9999):
                xs = [torch.ones(10_000, dtype=dt, device="cuda"), torch.ones(40, dtype=dt,
                                                                              device="cuda")]
                xs[0][place] = bad
                gq.gq_tensors_norm(gq.gq_tensors_create(xs), norm, norms=each)
                v = [float(norm), float(each[0]), float(each[1])]
                assert all(np.isnan(a) if np.isnan(bad) else a == np.inf for a in v[:2]), (dt, place)
                assert abs(v[2] - np.sqrt(40)) <= np.sqrt(40) * 2.0 ** -23


def _want(x, f, out):
    """The definition: the product in binary32, rounded to the output's type."""
    return (x.float() * torch.tensor(f, dtype=torch.float32, device=x.device)).to(out)


def _factor(norm, max_norm, eps, mul):
    top = float(np.float32(norm)) + float(np.float32(eps))
    m = float(np.float32(max_norm))
    c = 1.0 if top <= m else m / top
    return float(np.float32(c * float(np.float32(mul))))


def _bits(a, b):
    v = {4: torch.int32, 2: torch.int16}[a.element_size()]
    nan = torch.isnan(a) & torch.isnan(b)
    return bool(((a.view(v) == b.view(v)) | nan).all())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16", "mixed"])
@pytest.mark.parametrize("out", ["", "f32", "f16", "bf16", "mixed"])
def test_clip(gq, dt, out):
    kinds = ("bf16", "f32", "f16")
    for k, lengths in enumerate(LENGTHS):
        for gap in (0, 1):
            dts = [dt if dt != "mixed" else kinds[i % 3] for i in range(len(lengths))]
            odt = [out if out != "mixed" else kinds[i % 2] for i in range(len(lengths))]
            say("clip", dt, "into", out or "itself", "gap", gap, "case", k)
            for norm, top, eps, mul in ((2.0, 1.0, 1e-6, 1.0), (0.5, 1.0, 1e-6, 0.125),
                                        (3.7, 1.1, 0.0, 2.0 ** -3)):
                xs, flat = _make(lengths, dts, 200 + k, gap=gap)
                before = [x.clone() for x in xs]
                whole = {d: f.clone() for d, f in flat.items()}
                t = gq.gq_tensors_create(xs)
                nd = torch.tensor([norm], device="cuda")
                f = _factor(norm, top, eps, mul)
                if out:
                    ys, yflat = _make(lengths, odt, 300 + k, gap=gap)
                    ywhole = {d: b.clone() for d, b in yflat.items()}
                    gq.gq_tensors_clip(t, nd, top, eps=eps, in_mul=mul, out=gq.gq_tensors_create(ys))
                    assert all(_bits(flat[d], whole[d]) for d in flat), "the input changed"
                else:
                    ys, yflat, ywhole = xs, flat, whole
                    gq.gq_tensors_clip(t, nd, top, eps=eps, in_mul=mul)
                for i, (b, y) in enumerate(zip(before, ys)):
                    assert _bits(y, _want(b, f, y.dtype)), (dt, out, gap, k, i, f)
                for y in ys:
                    y.zero_()
                # and nothing between the tensors
                for d in yflat:
                    at = gap
                    for m, e in zip(lengths, odt if out else dts):
                        if e == d:
                            ywhole[d][at:at + m] = 0
                            at += m + gap
                    assert _bits(yflat[d], ywhole[d]), "wrote between the tensors"


def test_clip_borders(gq):
    """No clipping, the border itself, zero and infinite limits, NaN and
    infinite norms."""
    inf, nan = float("inf"), float("nan")
    x0 = torch.tensor([1.0, -2.5, 0.0, -0.0, inf, -inf, nan, 1e-40, 3e38], device="cuda")
    for norm, top, eps, mul in ((1.0, 1.0, 0.0, 1.0), (1.0, 1.0, 1e-6, 1.0), (0.0, 0.0, 0.0, 1.0),
                                (1.0, 0.0, 0.0, 1.0), (1e30, inf, 0.0, 0.5), (inf, inf, 0.0, 1.0),
                                (inf, 1.0, 1e-6, 1.0), (nan, 1.0, 1e-6, 1.0), (nan, inf, 0.0, 1.0),
                                (1e-45, 1e-45, 0.0, 1.0), (3e38, 1e-38, 0.0, 1.0)):
        f = _factor(norm, top, eps, mul) if norm == norm else nan
        for apart in (False, True):
            x, y = x0.clone(), torch.full_like(x0, 5.0)
            t = gq.gq_tensors_create([x])
            o = gq.gq_tensors_create([y]) if apart else None
            gq.gq_tensors_clip(t, torch.tensor([norm], device="cuda"), top, eps=eps, in_mul=mul, out=o)
            got, want = (y if apart else x), _want(x0, f, torch.float32)
            assert _bits(got, want), (norm, top, eps, mul, apart, got, want)


def test_refusals_on_live_lists(gq):
    a, b = torch.ones(100, device="cuda"), torch.ones(100, device="cuda", dtype=torch.bfloat16)
    norm = torch.ones(1, device="cuda")
    t = gq.gq_tensors_create([a[:40], a[50:]])
    with pytest.raises(gq.GQError, match="share memory"):
        gq.gq_tensors_create([a[:40], a[39:]])
    for other in ([b[:40]], [b[:40], b[40:91]], [b[:50], b[50:90]]):
        with pytest.raises(gq.GQError, match="other lengths"):
            gq.gq_tensors_clip(t, norm, 1.0, out=gq.gq_tensors_create(other))
    for other in ([a[:40], b[:50]], [a[10:50], b[:50]], [b[:40], a[40:90]]):
        with pytest.raises(gq.GQError, match="shares memory"):
            gq.gq_tensors_clip(t, norm, 1.0, out=gq.gq_tensors_create(other))
    assert bool((a == 1).all())
    # its own list as out is the list in place
    gq.gq_tensors_clip(t, norm * 2, 1.0, eps=0.0, out=t)
    assert bool((a[:40] == 0.5).all()) and bool((a[40:50] == 1).all())
    # lists that lie between each other's tensors
    gq.gq_tensors_clip(gq.gq_tensors_create([a[:10], a[20:30]]), norm, 1.0, eps=0.0, in_mul=4.0,
                       out=gq.gq_tensors_create([a[10:20], a[30:40]]))
    assert bool((a[10:20] == 2).all()) and bool((a[:10] == 0.5).all())
    gq.gq_tensors_destroy(t)
    with pytest.raises(ValueError):
        gq.gq_tensors_norm(t, norm)


def test_repeats_and_streams(gq):
    """Equal bits from call to call, on another stream than the tensors' own,
    and two lists of the same tensors at once on two streams."""
    xs, _ = _make([100_000, 3, 4096 * 50 + 1, 999], ["f32", "bf16", "f16", "f32"], 5)
    t, u = gq.gq_tensors_create(xs), gq.gq_tensors_create(xs)
    want = torch.empty(1, device="cuda")
    gq.gq_tensors_norm(t, want)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = torch.empty(50, device="cuda"), torch.empty(50, device="cuda")
    torch.cuda.synchronize()
    for i in range(50):
        gq.gq_tensors_norm(t, a[i:], stream=s1)
        with torch.cuda.stream(s2):
            gq.gq_tensors_norm(u, b[i:])
    torch.cuda.synchronize()
    assert bool((a == want).all()) and bool((b == want).all())


def test_captured(gq):
    """Norm and clip in one graph, replayed on new contents with eager calls
    of the same list between the replays."""
    xs, flat = _make([70_000, 5, 8192, 12_345], ["f32", "f32", "bf16", "f16"], 6)
    t = gq.gq_tensors_create(xs)
    norm, each = torch.zeros(1, device="cuda"), torch.zeros(4, device="cuda")
    eager = torch.zeros(1, device="cuda")
    gq.gq_tensors_norm(t, norm)                      # warm
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gq.gq_tensors_norm(t, norm, norms=each, in_mul=0.5)
        gq.gq_tensors_clip(t, norm, 1.0, in_mul=0.5)
    for k in range(5):
        for i, x in enumerate(xs):
            x.copy_(torch.randn(x.numel(), generator=torch.Generator().manual_seed(10 * k + i)))
        before = [x.clone() for x in xs]
        gq.gq_tensors_norm(t, eager, in_mul=0.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert float(norm) == float(eager)
        f = _factor(float(norm), 1.0, 1e-6, 0.5)
        for x, b, e in zip(xs, before, each):
            assert _bits(x, _want(b, f, x.dtype)), k
            _near(e, _norm64([b], 0.5), b.numel(), k)


def test_above_2_32_elements(gq):
    """A tensor whose elements' offsets pass 32 bits."""
    n = (1 << 32) + 4099
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    places = [0, 1, (1 << 31) - 1, (1 << 31), (1 << 32) - 1, 1 << 32, n - 1]
    for p in places:
        x[p] = 3.0
    t = gq.gq_tensors_create([x])
    norm = torch.empty(1, device="cuda")
    gq.gq_tensors_norm(t, norm)
    _near(norm[0], 3.0 * np.sqrt(len(places)), n, "norm")
    gq.gq_tensors_clip(t, torch.ones(1, device="cuda"), 0.5, eps=0.0)
    assert all(float(x[p]) == 1.5 for p in places)
    gq.gq_tensors_norm(t, norm)
    _near(norm[0], 1.5 * np.sqrt(len(places)), n, "norm after")


def test_most_tensors(gq):
    """2^20 tensors, every third one empty, through the C ABI."""
    import ctypes
    count = 1 << 20
    rng = np.random.default_rng(8)
    numel = rng.integers(1, 9, count).astype(np.int64)
    numel[::3] = 0
    numel[7] = 3 * TILE + 1
    at = np.concatenate([[0], np.cumsum(numel)])
    x = torch.randn(int(at[-1]), device="cuda")
    ptr = (x.data_ptr() + 4 * at[:-1]).astype(np.uint64)
    dt = np.zeros(count, np.int32)
    h = ctypes.c_void_p()
    assert gq.lib.gq_tensors_create(ptr.ctypes.data, numel.ctypes.data, dt.ctypes.data, count,
                                    ctypes.byref(h)) == gq.GQ_OK, gq.gq_last_error()
    norm, norms = torch.empty(1, device="cuda"), torch.full((count,), 7.0, device="cuda")
    assert gq.lib.gq_tensors_norm(h, 1.0, norm.data_ptr(), norms.data_ptr(), None) == gq.GQ_OK
    torch.cuda.synchronize()
    _near(norm[0], _norm64([x]), x.numel(), "all")
    sums = np.concatenate([[0.0], np.cumsum(x.double().cpu().numpy() ** 2)])
    want = np.sqrt(np.diff(sums[at]))
    # (the running sum's rounding, of up to its last value)
    off = np.abs(norms.double().cpu().numpy() - want)
    slack = sums[-1] * 2.0 ** -52 * x.numel() ** 0.5
    assert np.all(off <= want * 2.0 ** -23 + slack / np.maximum(want, 1e-3))
    assert bool((norms[::3] == 0).all())
    before = x.clone()
    assert gq.lib.gq_tensors_clip(h, norm.data_ptr(), 1.0, 0.0, 1.0, None, None) == gq.GQ_OK
    torch.cuda.synchronize()
    assert _bits(x, _want(before, _factor(float(norm), 1.0, 0.0, 1.0), torch.float32))
    assert gq.lib.gq_tensors_destroy(h) == gq.GQ_OK


def test_norm_inside_a_list(gq):
    """A norm in a tensor that the call writes, or that its norm is taken of, is
    refused before anything runs; one between the tensors, or in a list that
    is only read, is not."""
    flat = torch.arange(1, 20_001, dtype=torch.float32, device="cuda")
    before = flat.clone()
    t = gq.gq_tensors_create([flat[4:9000], flat[9004:19_000]])
    two = torch.empty(2, device="cuda")
    for p in (flat[4:5], flat[8999:9000], flat[9004:9005], flat[18_999:19_000]):
        for call in (lambda: gq.gq_tensors_norm(t, p), lambda: gq.gq_tensors_clip(t, p, 1.0)):
            with pytest.raises(gq.GQError, match="lies in a tensor"):
                call()
    for p in (flat[3:5], flat[9003:9005], flat[18_999:19_001]):
        with pytest.raises(gq.GQError, match="lies in a tensor"):
            gq.gq_tensors_norm(t, two, norms=p)
    for p in (two[:1], two[1:]):
        with pytest.raises(gq.GQError, match="one of norms"):
            gq.gq_tensors_norm(t, p, norms=two)
    torch.cuda.synchronize()
    assert torch.equal(flat, before)
    # between and behind the tensors
    gq.gq_tensors_norm(t, flat[9002:9003], norms=flat[19_000:19_002])
    want = [_norm64([before[4:9000]]), _norm64([before[9004:19_000]])]
    for got, w, n in ((flat[9002], np.hypot(*want), 18_992), (flat[19_000], want[0], 8996),
                      (flat[19_001], want[1], 9996)):
        _near(got, w, n, "beside the tensors")
    # in a tensor that is only read
    y = torch.empty(18_992, device="cuda")
    gq.gq_tensors_clip(t, flat[4:5], 2.0, eps=0.0,
                       out=gq.gq_tensors_create([y[:8996], y[8996:]]))
    f = _factor(5.0, 2.0, 0.0, 1.0)
    assert _bits(y, _want(torch.cat([before[4:9000], before[9004:19_000]]), f, torch.float32))
