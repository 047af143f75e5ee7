"""Host checks of the gq_mx4_* calls, without a GPU: argument errors are
returned before the device is touched, and the binding refuses tensors that
the library would overrun."""
import ctypes

import numpy as np
import pytest
import torch

from tests import mx4_ref as ref

GOOD = 0x10000


@pytest.fixture(scope="module")
def gq():
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _arr(vals):
    return ctypes.cast((ctypes.c_void_p * len(vals))(*vals), ctypes.c_void_p)


def test_sizes(gq):
    for rows, cols in ((1, 1), (1, 32), (3, 33), (5, 1000), (1 << 20, 7)):
        nb = ref.blocks(cols)
        assert gq.gq_mx4_sizes(rows, cols) == (rows * nb, rows * nb * 16)
    for rows, cols in ((0, 1), (1, 0), (-1, 4), ((1 << 40) + 1, 1), (1 << 36, 1), (1 << 21, 1 << 20)):
        with pytest.raises(gq.GQError) as e:
            gq.gq_mx4_sizes(rows, cols)
        assert e.value.status == gq.GQ_ERR_INVALID


def _call(fn, names, good):
    def call(**kw):
        a = dict(zip(names, good))
        a.update(kw)
        return fn(*(a[n] for n in names))
    return call


def test_quantize_refusals(gq):
    p = _arr([GOOD] * 2)
    call = _call(gq.lib.gq_mx4_quantize,
                 ("x", "W", "dt", "mul", "rows", "cols", "ld", "t", "s", "q", "st"),
                 (p, 2, gq.GQ_F32, 1.0, 4, 40, 40, 0, p, p, None))
    bad = [dict(W=0), dict(W=65), dict(dt=3), dict(dt=-1), dict(mul=0.0), dict(mul=float("nan")),
           dict(rows=0), dict(cols=0), dict(ld=39), dict(rows=1 << 40), dict(x=None), dict(s=None),
           dict(q=None), dict(x=_arr([GOOD, 0])), dict(cols=1 << 36, ld=1 << 36, rows=32),
           # one element per 32-code block
           dict(cols=1, ld=1, rows=1 << 36), dict(rows=1, cols=1 << 36, t=1)]
    for kw in bad:
        assert call(**kw) == gq.GQ_ERR_INVALID, kw
        assert gq.gq_last_error().startswith("gq_mx4_quantize"), kw
    for kw in (dict(x=_arr([GOOD, GOOD + 8])), dict(q=_arr([GOOD + 4, GOOD]))):
        assert call(**kw) == gq.GQ_ERR_ALIGN, kw


def test_reduce_refusals(gq):
    p = _arr([GOOD] * 2)
    call = _call(gq.lib.gq_mx4_reduce_dequant, ("q", "s", "W", "rows", "cols", "r", "st"),
                 (p, p, 2, 3, 40, GOOD, None))
    for kw in (dict(W=0), dict(W=65), dict(rows=0), dict(cols=-1), dict(q=None), dict(s=None),
               dict(r=None), dict(rows=1 << 36, cols=1)):
        assert call(**kw) == gq.GQ_ERR_INVALID, kw
    assert call(r=GOOD + 8) == gq.GQ_ERR_ALIGN
    assert call(q=_arr([GOOD, GOOD + 1])) == gq.GQ_ERR_ALIGN
    call = _call(gq.lib.gq_mx4_reduce_requantize,
                 ("q", "s", "W", "rows", "cols", "r", "so", "qo", "st"),
                 (p, p, 2, 3, 40, None, GOOD, GOOD, None))
    for kw in (dict(so=None), dict(qo=None), dict(W=-1)):
        assert call(**kw) == gq.GQ_ERR_INVALID, kw
    assert call(r=GOOD + 4) == gq.GQ_ERR_ALIGN
    assert call(qo=GOOD + 8) == gq.GQ_ERR_ALIGN


def test_product_refusals(gq):
    m, n, k = 40, 50, 30000
    need = gq.gq_mx4_product_workspace(m, n, k)
    assert need > 0 and need % (4 * m * n) == 0
    assert gq.gq_mx4_product_workspace(8192, 8192, 8192) == 0
    assert gq.gq_mx4_product_workspace(1, 1, 32) == 0
    call = _call(gq.lib.gq_mx4_product,
                 ("a", "sa", "b", "sb", "m", "n", "k", "dt", "add", "c", "ldc", "ws", "wn", "st"),
                 (GOOD, GOOD, GOOD, GOOD, m, n, k, gq.GQ_F32, 0, GOOD, n, None, 0, None))
    for kw in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(c=None), dict(m=0),
               dict(n=0), dict(k=0), dict(k=(1 << 24) + 1), dict(m=1 << 29), dict(ldc=n - 1),
               dict(dt=5), dict(dt=gq.GQ_BF16, add=1), dict(dt=gq.GQ_F16, add=1),
               dict(m=1 << 20, n=1 << 20)):
        assert call(**kw) == gq.GQ_ERR_INVALID, kw
    for kw in (dict(a=GOOD + 8), dict(b=GOOD + 4), dict(c=GOOD + 2), dict(dt=gq.GQ_F16, c=GOOD + 1),
               dict(ws=GOOD + 8, wn=need)):
        assert call(**kw) == gq.GQ_ERR_ALIGN, kw
    assert call(ws=GOOD, wn=need - 1) == gq.GQ_ERR_CAPACITY
    for bad in ((0, 1, 1), (1, 1, 0), (1 << 29, 1, 1)):
        with pytest.raises(gq.GQError):
            gq.gq_mx4_product_workspace(*bad)


class Fake:
    """What the guards read of a tensor on the device."""

    def __init__(self, shape, dtype, stride=None, cuda=True, device=0):
        self.shape = shape if isinstance(shape, tuple) else (shape,)
        self.dtype, self.is_cuda, self._device = dtype, cuda, device
        dense = []
        for d in reversed(self.shape):
            dense.insert(0, dense[0] * self.shape[len(self.shape) - len(dense)] if dense else 1)
        self._stride = stride or tuple(dense)
        self._dense = self._stride == tuple(dense)

    def stride(self):
        return self._stride

    def numel(self):
        return int(np.prod(self.shape))

    def is_contiguous(self):
        return self._dense

    def data_ptr(self):
        return GOOD

    def get_device(self):
        return self._device


class Reached(Exception):
    pass


@pytest.fixture()
def stub(gq, monkeypatch):
    class Lib:
        def __getattr__(self, name):
            def f(*a):
                raise Reached(name)
            return f
    monkeypatch.setattr(gq, "lib", Lib())
    monkeypatch.setattr(gq, "_current_device", lambda: 0)
    monkeypatch.setattr(gq, "_stream", lambda s: ctypes.c_void_p(0))
    return gq


F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8


def test_binding_guards(stub):
    gq = stub
    x, s, q = Fake((4, 40), F32), Fake(8, U8), Fake(128, U8)
    r = Fake(160, F32)
    good = [lambda: gq.gq_mx4_quantize([x, x], [s, s], [q, q]),
            lambda: gq.gq_mx4_quantize([Fake(100, BF16)], [s], [q]),
            lambda: gq.gq_mx4_quantize([Fake((4, 40), F32, (50, 1))], [s], [q]),
            lambda: gq.gq_mx4_quantize([x], [Fake(40, U8)], [Fake(640, U8)], transpose=True),
            lambda: gq.gq_mx4_reduce_dequant([q], [s], 4, 40, r),
            lambda: gq.gq_mx4_reduce_requantize([q, q], [s, s], 4, 40, s, q, r_out=r),
            lambda: gq.gq_mx4_product(q, s, q, s, 40, Fake((4, 4), BF16)),
            lambda: gq.gq_mx4_product(q, s, q, s, 40, Fake((4, 4), F32, (9, 1)), accumulate=True,
                                      workspace=Fake(0, U8))]
    for f in good:
        with pytest.raises(Reached):
            f()
    bad = [lambda: gq.gq_mx4_quantize([], [], []),
           lambda: gq.gq_mx4_quantize([x], [Fake(7, U8)], [q]),
           lambda: gq.gq_mx4_quantize([x], [s], [Fake(127, U8)]),
           lambda: gq.gq_mx4_quantize([x], [s], [q], transpose=True),
           lambda: gq.gq_mx4_quantize([x], [s], [Fake(128, torch.int8)]),
           lambda: gq.gq_mx4_quantize([x, Fake((4, 41), F32)], [s, s], [q, q]),
           lambda: gq.gq_mx4_quantize([x, Fake((4, 40), BF16)], [s, s], [q, q]),
           lambda: gq.gq_mx4_quantize([Fake((4, 40), torch.int32)], [s], [q]),
           lambda: gq.gq_mx4_quantize([Fake((4, 40), F32, (1, 4))], [s], [q]),
           lambda: gq.gq_mx4_quantize([Fake((4, 40), F32, (0, 1))], [s], [q]),
           lambda: gq.gq_mx4_quantize([Fake((2, 2, 40), F32)], [s], [q]),
           lambda: gq.gq_mx4_quantize([Fake((0, 40), F32)], [s], [q]),
           lambda: gq.gq_mx4_quantize([Fake((4, 40), F32, cuda=False)], [s], [q]),
           lambda: gq.gq_mx4_quantize([Fake((4, 40), F32, device=1)], [s], [q]),
           lambda: gq.gq_mx4_reduce_dequant([q], [s], 4, 40, Fake(159, F32)),
           lambda: gq.gq_mx4_reduce_dequant([q], [s], 4, 65, r),
           lambda: gq.gq_mx4_reduce_dequant([q], [s], 0, 40, r),
           lambda: gq.gq_mx4_reduce_dequant([q], [s], 4, 40, Fake(160, BF16)),
           lambda: gq.gq_mx4_reduce_requantize([q], [s], 4, 40, Fake(7, U8), q),
           lambda: gq.gq_mx4_reduce_requantize([q], [s, s], 4, 40, s, q),
           lambda: gq.gq_mx4_product(q, s, q, s, 65, Fake((4, 4), F32)),
           lambda: gq.gq_mx4_product(q, s, q, s, 40, Fake((5, 4), F32)),
           lambda: gq.gq_mx4_product(q, s, q, s, 40, Fake((4, 5), F32)),
           lambda: gq.gq_mx4_product(q, s, q, s, 0, Fake((4, 4), F32)),
           lambda: gq.gq_mx4_product(q, s, q, s, 40, Fake((4, 4), torch.float64)),
           lambda: gq.gq_mx4_product(q, s, q, s, 40, Fake((4, 4), F32), workspace=Fake(9, F32))]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail("call %d was accepted" % i)


def test_reference_rounds_to_nearest():
    """The reference's codes are the nearest values, ties to the even code."""
    x = np.linspace(-7.99, 7.99, 4001).astype(np.float32)
    x = np.concatenate([np.array([4.0], np.float32), x])
    for v in x:
        block = np.full((1, 32), 4.0, np.float32)
        block[0, 0] = v
        s, q = ref.quantize(block)
        assert s[0, 0] == 127
        d = np.abs(ref.VALUES[:8] - abs(float(v)))
        best = np.flatnonzero(d == d.min())
        want = best[0] if len(best) == 1 else best[best % 2 == 0][0]
        assert (q[0, 0, 0] & 7) == want and bool(q[0, 0, 0] & 8) == bool(v < 0)
