"""The 4-bit format's conversions over all of what they take: every code at
every scale byte, every binary32 magnitude below 8 at one scale, the ends of
the rounding intervals and their neighbours at every scale, and every fp16 and
bf16 value."""
import numpy as np
import pytest
import torch

from tests import mx4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).reshape(-1)).cuda()


def _buffers(gq, rows, cols):
    n, b = gq.gq_mx4_sizes(rows, cols)
    return (torch.full((k,), 0xA5, dtype=torch.uint8, device="cuda") for k in (n, b))


def _quantized(gq, x):
    rows, cols = x.shape
    s, q = _buffers(gq, rows, cols)
    gq.gq_mx4_quantize([x], [s], [q])
    return s.cpu().numpy().reshape(rows, -1), q.cpu().numpy().reshape(rows, -1, 16)


def test_every_code_at_every_scale(gq):
    c = np.tile(np.arange(16, dtype=np.uint8), 2)
    q = np.broadcast_to(c[0::2] | c[1::2] << 4, (256, 1, 16)).copy()
    s = np.arange(256, dtype=np.uint8).reshape(256, 1)
    out = torch.zeros(256 * 32, device="cuda")
    gq.gq_mx4_reduce_dequant([_dev(q)], [_dev(s)], 256, 32, out)
    with np.errstate(over="ignore"):
        want = ref.reduce([s], [q], 32)
    got = out.cpu().numpy().reshape(256, 32)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(want[255]).all()
    # (a sum that starts at +0 has no -0)
    assert np.array_equal(got[:255].view(np.uint32), want[:255].view(np.uint32))


def test_interval_ends_at_every_scale(gq):
    """The ends of the intervals that round to each magnitude, the magnitudes,
    and both neighbours of each in binary32, at every scale that a finite
    maximum gives; one element of each block sets the scale."""
    ends = np.array([e for e, _ in ref.ENDS] + [0.5, 1, 1.5, 2, 3, 4, 6, 7])
    rows = []
    for s in range(253):
        v = np.ldexp(ends, s - 127).astype(np.float32)
        assert np.array_equal(v.astype(np.float64), np.ldexp(ends, s - 127))
        near = [v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf))]
        most = np.ldexp(2 - 2.0 ** -23, s - 125)        # the largest below 8
        v = np.concatenate(near + [[most]]).astype(np.float32)
        v = np.concatenate([v, -v, [0.0, -0.0]])
        v = np.concatenate([v, np.zeros(-v.size % 31, np.float32)]).reshape(-1, 31)
        top = np.full((v.shape[0], 1), np.ldexp(4.0, s - 127), np.float32)
        rows.append(np.concatenate([top, v], 1).astype(np.float32))
    x = np.concatenate(rows)
    s_ref, q_ref = ref.quantize(x)
    assert set(s_ref.reshape(-1).tolist()) == set(range(253))
    s, q = _quantized(gq, torch.from_numpy(x).cuda())
    assert np.array_equal(s, s_ref)
    bad = np.argwhere(q != q_ref)
    assert bad.size == 0, (x[bad[0][0]], q[bad[0][0]], q_ref[bad[0][0]])


@pytest.mark.parametrize("sign", [0, 1])
def test_every_magnitude_below_eight(gq, sign):
    """All 0x41000000 bit patterns below that of 8.0, 31 a block beside a 4.0
    (so that the scale is 1), against comparisons with the intervals' ends."""
    end = 0x41000000
    step = 31 << 21
    blocks = step // 31
    s, q = _buffers(gq, blocks, 32)
    x = torch.empty(blocks, 32, dtype=torch.int32, device="cuda")
    for lo in range(0, end, step):
        say("patterns from", hex(lo), "sign", sign)
        v = torch.arange(lo, lo + step, dtype=torch.int64, device="cuda").clamp(max=end - 1)
        x[:, 0] = 0x40800000
        x[:, 1:] = v.to(torch.int32).view(blocks, 31)
        a = x.view(torch.float32)
        code = torch.zeros(blocks, 32, dtype=torch.uint8, device="cuda")
        for e, up in ref.ENDS:
            code += (a >= e) if up else (a > e)
        if sign:
            a = -a
            code += 8
        gq.gq_mx4_quantize([a], [s], [q])
        assert bool((s == 127).all())
        assert torch.equal(q.view(blocks, 16), code[:, 0::2] | code[:, 1::2] << 4)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_every_16_bit_value(gq, dt):
    """Every bit pattern among its neighbours, and among random others (blocks
    of finite ones, as an inf or a NaN clears its block)."""
    rng = np.random.default_rng(41)
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    inf = 0x7C00 if dt == "f16" else 0x7F80
    finite = bits[(bits & 0x7FFF) < inf]
    finite = finite[:finite.size // 32 * 32]
    t = torch.float16 if dt == "f16" else torch.bfloat16
    for v in [bits] + [rng.permutation(finite) for _ in range(4)]:
        x = torch.from_numpy(v.view(np.int16).copy()).cuda().view(t).view(-1, 32)
        s, q = _quantized(gq, x)
        s_ref, q_ref = ref.quantize(x.float().cpu().numpy())
        assert np.array_equal(s, s_ref) and np.array_equal(q, q_ref)
