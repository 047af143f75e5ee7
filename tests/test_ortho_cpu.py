"""Host checks of the gq_ortho_* calls, without a GPU: argument errors are
returned before the device is touched."""
import ctypes

import numpy as np
import pytest
import torch

GOOD = 0x10000


@pytest.fixture(scope="module")
def gq():
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _create(gq, off=(0, 100), rows=(10, 4), cols=(10, 5), n=2, steps=5, coef=None, eps=1e-7,
            out_mul=None, out=True):
    arrays = [np.array(v, np.int64) if v is not None else None for v in (off, rows, cols)]
    c = np.array(coef, np.float32) if coef is not None else None
    m = np.array(out_mul, np.float32) if out_mul is not None else None
    h = ctypes.c_void_p(1)
    st = gq.lib.gq_ortho_create(*(a.ctypes.data if a is not None else None for a in arrays), n,
                                steps, c.ctypes.data if c is not None else None, eps,
                                m.ctypes.data if m is not None else None,
                                ctypes.byref(h) if out else None)
    if out and st != gq.GQ_OK:
        assert not h.value, "the handle must be cleared on an error"
    return st


def test_create_refusals(gq):
    nan, inf = float("nan"), float("inf")
    bad = [dict(out=False), dict(off=None), dict(rows=None), dict(cols=None), dict(n=0),
           dict(n=(1 << 20) + 1), dict(steps=0), dict(steps=17), dict(eps=-1.0), dict(eps=nan),
           dict(eps=inf), dict(coef=[1, 2, inf] * 5), dict(out_mul=[1.0, nan]),
           dict(rows=(10, 0)), dict(cols=(-1, 5)), dict(off=(0, 99)), dict(off=(-1, 100)),
           dict(rows=(10, (1 << 22) + 1)), dict(rows=(10, 40000), cols=(10, 40000)),
           dict(off=(0, (1 << 40) - 5))]
    for kw in bad:
        assert _create(gq, **kw) == gq.GQ_ERR_INVALID, kw
        assert gq.gq_last_error().startswith("gq_ortho_create"), kw


def test_step_refusals(gq):
    names = ("p", "g", "dt", "mul", "m", "mu", "nest", "odt", "out", "st")
    good = dict(zip(names, (None, GOOD, gq.GQ_F32, 1.0, GOOD, 0.9, 1, gq.GQ_BF16, GOOD, None)))

    def call(**kw):
        a = dict(good)
        a.update(kw)
        return gq.lib.gq_ortho_step(*(a[n] for n in names))

    for kw in (dict(dt=3), dict(mul=0.0), dict(mul=float("inf")), dict(odt=gq.GQ_F32), dict(odt=9),
               dict(g=None), dict(out=None), dict(mu=-0.1), dict(mu=float("nan"))):
        assert call(**kw) == gq.GQ_ERR_INVALID, kw
    for kw in (dict(g=GOOD + 8), dict(out=GOOD + 4), dict(m=GOOD + 8)):
        assert call(**kw) == gq.GQ_ERR_ALIGN, kw
    assert call() == gq.GQ_ERR_INVALID and "plan is NULL" in gq.gq_last_error()
    assert gq.lib.gq_ortho_info(None, None, None, None, None) == gq.GQ_ERR_INVALID
    assert gq.lib.gq_ortho_destroy(None) == gq.GQ_OK


def test_binding_guards(gq, monkeypatch):
    for kw in (dict(shapes=[]), dict(shapes=[1, 2]), dict(shapes=[(1, 2, 3)]),
               dict(shapes=[(2, 3)], offsets=[0, 6]), dict(shapes=[(2, 3)], coef=[(1, 2, 3)] * 4),
               dict(shapes=[(2, 3)], out_mul=[1.0, 2.0])):
        with pytest.raises(ValueError):
            gq.gq_ortho_create(**kw)

    class Fake:
        def __init__(self, n, dtype, cuda=True, dense=True, device=0):
            self.n, self.dtype, self.is_cuda, self.dense, self.device = n, dtype, cuda, dense, device

        def numel(self):
            return self.n

        def is_contiguous(self):
            return self.dense

        def get_device(self):
            return self.device

        def data_ptr(self):
            return GOOD

    class Reached(Exception):
        pass

    class Lib:
        def __getattr__(self, name):
            def f(*a):
                raise Reached(name)
            return f

    monkeypatch.setattr(gq, "lib", Lib())
    monkeypatch.setattr(gq, "_current_device", lambda: 0)
    monkeypatch.setattr(gq, "_stream", lambda s: ctypes.c_void_p(0))
    plan = gq.Ortho.__new__(gq.Ortho)
    plan.handle, plan.n = ctypes.c_void_p(1), 100
    F32, F16, BF = torch.float32, torch.float16, torch.bfloat16
    g, o, m = Fake(100, F32), Fake(100, BF), Fake(100, F32)
    for f in (lambda: gq.gq_ortho_step(plan, g, o), lambda: gq.gq_ortho_step(plan, g, o, momentum=m),
              lambda: gq.gq_ortho_step(plan, Fake(100, BF), Fake(200, F16))):
        with pytest.raises(Reached):
            f()
    dead = gq.Ortho.__new__(gq.Ortho)
    for f in (lambda: gq.gq_ortho_step(None, g, o), lambda: gq.gq_ortho_step(dead, g, o),
              lambda: gq.gq_ortho_step(plan, Fake(99, F32), o),
              lambda: gq.gq_ortho_step(plan, g, Fake(99, BF)),
              lambda: gq.gq_ortho_step(plan, g, Fake(100, F32)),
              lambda: gq.gq_ortho_step(plan, Fake(100, torch.int8), o),
              lambda: gq.gq_ortho_step(plan, g, o, momentum=Fake(99, F32)),
              lambda: gq.gq_ortho_step(plan, g, o, momentum=Fake(100, F16)),
              lambda: gq.gq_ortho_step(plan, Fake(100, F32, dense=False), o),
              lambda: gq.gq_ortho_step(plan, Fake(100, F32, cuda=False), o),
              lambda: gq.gq_ortho_step(plan, Fake(100, F32, device=1), o)):
        with pytest.raises((ValueError, TypeError)):
            f()
    plan.handle = ctypes.c_void_p()
