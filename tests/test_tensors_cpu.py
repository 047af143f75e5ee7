"""Host checks of the gq_tensors_* calls, without a GPU: argument errors are
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


def _create(gq, x=(GOOD, GOOD + 4096), numel=(100, 7), dt=(0, 0), count=2, out=True):
    px = np.array([p or 0 for p in x], np.uint64) if x is not None else None
    n = np.array(numel, np.int64) if numel is not None else None
    t = np.array(dt, np.int32) if dt is not None else None
    h = ctypes.c_void_p(1)
    st = gq.lib.gq_tensors_create(*(a.ctypes.data if a is not None else None for a in (px, n, t)),
                                  count, ctypes.byref(h) if out else None)
    if out and st != gq.GQ_OK:
        assert not h.value, "the handle must be cleared on an error"
    return st


def test_create_refusals(gq):
    bad = [dict(out=False), dict(x=None), dict(numel=None), dict(dt=None), dict(count=0),
           dict(count=-1), dict(count=(1 << 20) + 1), dict(dt=(0, 3)), dict(dt=(-1, 0)),
           dict(numel=(-1, 7)), dict(numel=(100, (1 << 36) - 99)), dict(numel=((1 << 62), 1 << 62)),
           dict(x=(GOOD, None)), dict(x=(GOOD, GOOD)), dict(x=(GOOD, GOOD + 396)),
           dict(x=(GOOD + 24, GOOD)), dict(x=(GOOD, GOOD + 198), dt=(1, 1))]
    for kw in bad:
        assert _create(gq, **kw) == gq.GQ_ERR_INVALID, kw
        assert gq.gq_last_error().startswith("gq_tensors_create"), kw
    for kw in (dict(x=(GOOD + 2, GOOD + 4096)), dict(x=(GOOD, GOOD + 4097), dt=(0, 2)),
               dict(x=(GOOD, GOOD + 4098))):
        assert _create(gq, **kw) == gq.GQ_ERR_ALIGN, kw


def test_norm_and_clip_refusals(gq):
    nan, inf = float("nan"), float("inf")
    L = gq.lib
    for mul in (0.0, -1.0, nan, inf):
        assert L.gq_tensors_norm(None, mul, GOOD, None, None) == gq.GQ_ERR_INVALID
        assert L.gq_tensors_clip(None, GOOD, 1.0, 0.0, mul, None, None) == gq.GQ_ERR_INVALID
        assert "in_mul" in gq.gq_last_error()
    assert L.gq_tensors_norm(None, 1.0, None, None, None) == gq.GQ_ERR_INVALID
    assert L.gq_tensors_norm(None, 1.0, GOOD + 2, None, None) == gq.GQ_ERR_ALIGN
    assert L.gq_tensors_norm(None, 1.0, GOOD, GOOD + 1, None) == gq.GQ_ERR_ALIGN
    assert L.gq_tensors_norm(None, 1.0, GOOD, None, None) == gq.GQ_ERR_INVALID
    assert "list is NULL" in gq.gq_last_error()
    for top, eps in ((-1.0, 0.0), (nan, 0.0), (1.0, -1e-6), (1.0, nan), (1.0, inf)):
        assert L.gq_tensors_clip(None, GOOD, top, eps, 1.0, None, None) == gq.GQ_ERR_INVALID
        assert "list" not in gq.gq_last_error()
    assert L.gq_tensors_clip(None, None, 1.0, 0.0, 1.0, None, None) == gq.GQ_ERR_INVALID
    assert L.gq_tensors_clip(None, GOOD + 2, 1.0, 0.0, 1.0, None, None) == gq.GQ_ERR_ALIGN
    assert L.gq_tensors_clip(None, GOOD, 1.0, 0.0, 1.0, None, None) == gq.GQ_ERR_INVALID
    assert "list is NULL" in gq.gq_last_error()
    assert L.gq_tensors_info(None, None, None, None) == gq.GQ_ERR_INVALID
    assert L.gq_tensors_destroy(None) == gq.GQ_OK


class Fake:
    """What the guards read of a tensor."""

    def __init__(self, shape, dtype, cuda=True, dense=True, device=0, ld=None):
        self.shape = (shape,) if isinstance(shape, int) else tuple(shape)
        self.dtype, self.is_cuda, self.dense, self.device = dtype, cuda, dense, device
        self.ld = ld

    def numel(self):
        return int(np.prod(self.shape))

    def is_contiguous(self):
        return self.dense

    def get_device(self):
        return self.device

    def data_ptr(self):
        return GOOD

    def stride(self):
        return (1,) if len(self.shape) == 1 else (self.ld or self.shape[1], 1)


class Reached(Exception):
    pass


class Lib:
    def __getattr__(self, name):
        def f(*a):
            raise Reached(name)
        return f


@pytest.fixture()
def stub(gq, monkeypatch):
    monkeypatch.setattr(gq, "lib", Lib())
    monkeypatch.setattr(gq, "_current_device", lambda: 0)
    monkeypatch.setattr(gq, "_stream", lambda s: ctypes.c_void_p(0))
    return gq


F32, F16, BF, I64 = torch.float32, torch.float16, torch.bfloat16, torch.int64


def test_binding_guards(stub):
    gq = stub
    ok = [Fake(10, F32), Fake(0, F16), Fake((3, 4), BF)]
    with pytest.raises(Reached):
        gq.gq_tensors_create(ok)
    for xs in ([], None, Fake(10, F32), [Fake(10, F32), None], [Fake(10, F32, cuda=False)],
               [Fake(10, F32, dense=False)], [Fake(10, F32, device=1)], [Fake(10, I64)],
               [Fake(10, torch.float64)]):
        with pytest.raises((ValueError, TypeError)):
            gq.gq_tensors_create(xs)
    t = gq.Tensors.__new__(gq.Tensors)
    t.handle, t.count = ctypes.c_void_p(1), 3
    dead = gq.Tensors.__new__(gq.Tensors)
    one, three = Fake(1, F32), Fake(3, F32)
    for f in (lambda: gq.gq_tensors_norm(t, one), lambda: gq.gq_tensors_norm(t, one, norms=three),
              lambda: gq.gq_tensors_clip(t, one, 1.0), lambda: gq.gq_tensors_clip(t, one, 1.0, out=t)):
        with pytest.raises(Reached):
            f()
    for f in (lambda: gq.gq_tensors_norm(None, one), lambda: gq.gq_tensors_norm(dead, one),
              lambda: gq.gq_tensors_norm(t, Fake(0, F32)), lambda: gq.gq_tensors_norm(t, Fake(1, F16)),
              lambda: gq.gq_tensors_norm(t, one, norms=Fake(2, F32)),
              lambda: gq.gq_tensors_norm(t, one, norms=Fake(3, BF)),
              lambda: gq.gq_tensors_clip(dead, one, 1.0),
              lambda: gq.gq_tensors_clip(t, Fake(1, F32, cuda=False), 1.0),
              lambda: gq.gq_tensors_clip(t, one, 1.0, out=dead),
              lambda: gq.gq_tensors_clip(t, one, 1.0, out=[one])):
        with pytest.raises((ValueError, TypeError)):
            f()
    t.handle = ctypes.c_void_p()


def test_embed_refusals(gq):
    names = ("idx", "ib", "n", "table", "dt", "rows", "cols", "ld", "mul", "odt", "out", "ldo", "st")
    good = dict(zip(names, (GOOD, 8, 5, GOOD, 0, 9, 16, 16, 1.0, 2, GOOD, 16, None)))

    def call(**kw):
        a = dict(good)
        a.update(kw)
        return gq.lib.gq_embed(*(a[n] for n in names))

    for kw in (dict(n=-1), dict(n=(1 << 30) + 1), dict(rows=0), dict(rows=(1 << 30) + 1),
               dict(cols=0), dict(cols=(1 << 24) + 1), dict(dt=3), dict(odt=-1),
               dict(mul=float("nan")), dict(mul=float("inf")), dict(ib=2), dict(idx=None),
               dict(table=None), dict(out=None), dict(ld=15), dict(ldo=15), dict(ld=1 << 37),
               dict(ldo=1 << 38)):
        assert call(**kw) == gq.GQ_ERR_INVALID, kw
        assert gq.gq_last_error().startswith("gq_embed"), kw
    for kw in (dict(idx=GOOD + 4), dict(idx=GOOD + 2, ib=4), dict(table=GOOD + 2),
               dict(out=GOOD + 1)):
        assert call(**kw) == gq.GQ_ERR_ALIGN, kw
    # no tokens: nothing to read or write
    assert call(n=0, idx=None, out=None) == gq.GQ_OK


def test_embed_grad_refusals(gq):
    names = ("idx", "ib", "n", "dy", "dt", "ldy", "mul", "skip", "rows", "cols", "odt", "add",
             "grad", "ldg", "ws", "wn", "st")
    need = gq.gq_embed_grad_workspace(5, 9, 16)
    good = dict(zip(names, (GOOD, 4, 5, GOOD, 2, 16, 1.0, -1, 9, 16, 0, 0, GOOD, 16, GOOD, need,
                            None)))

    def call(**kw):
        a = dict(good)
        a.update(kw)
        return gq.lib.gq_embed_grad(*(a[n] for n in names))

    for kw in (dict(n=-1), dict(rows=0), dict(cols=0), dict(dt=7), dict(odt=5), dict(odt=1, add=1),
               dict(odt=2, add=1), dict(mul=float("inf")), dict(ib=1), dict(idx=None),
               dict(dy=None), dict(grad=None), dict(ws=None), dict(ldy=15), dict(ldg=15)):
        assert call(**kw) == gq.GQ_ERR_INVALID, kw
        assert gq.gq_last_error().startswith("gq_embed_grad"), kw
    for kw in (dict(idx=GOOD + 2), dict(dy=GOOD + 1), dict(grad=GOOD + 2), dict(ws=GOOD + 8)):
        assert call(**kw) == gq.GQ_ERR_ALIGN, kw
    assert call(wn=need - 1) == gq.GQ_ERR_CAPACITY
    assert call(n=0, idx=None, dy=None, add=1) == gq.GQ_OK
    assert gq.lib.gq_embed_grad_workspace(5, 9, 16, None) == gq.GQ_ERR_INVALID
    for n, r, c in ((-1, 9, 16), (5, 0, 16), (5, 9, 0), (1 << 31, 9, 16), (5, 1 << 31, 16)):
        with pytest.raises(gq.GQError):
            gq.gq_embed_grad_workspace(n, r, c)


def test_embed_binding_guards(stub):
    gq = stub
    idx, table, out = Fake((2, 3), I64), Fake((9, 16), F32, ld=20), Fake((6, 16), BF, ld=17)
    dy, grad, ws = Fake((6, 16), BF), Fake((9, 16), F32), Fake(1 << 20, torch.uint8)
    none = Fake((0,), torch.int32)
    for f in (lambda: gq.gq_embed(idx, table, out),
              lambda: gq.gq_embed(Fake(1, torch.int32), table, Fake(16, F16)),
              lambda: gq.gq_embed(none, table, Fake((0, 16), BF)),
              lambda: gq.gq_embed_grad(idx, dy, grad, ws),
              lambda: gq.gq_embed_grad(none, Fake((0, 16), BF), grad, ws, skip=3)):
        with pytest.raises(Reached):
            f()
    bad_idx = (Fake((2, 3), F32), Fake((2, 3), I64, cuda=False), Fake((2, 3), I64, dense=False),
               Fake((2, 3), I64, device=1), Fake(5, I64), none)
    bad_rows = (Fake((6, 15), BF), Fake((5, 16), BF), Fake((6, 16), I64),
                Fake((6, 16), BF, cuda=False), Fake((6, 16), BF, device=1), Fake((2, 3, 16), BF),
                Fake((6, 16), BF, ld=15), Fake((0, 16), BF))
    for i in bad_idx:
        for f in (lambda: gq.gq_embed(i, table, out), lambda: gq.gq_embed_grad(i, dy, grad, ws)):
            with pytest.raises((ValueError, TypeError)):
                f()
    for t in bad_rows:
        for f in (lambda: gq.gq_embed(idx, table, t), lambda: gq.gq_embed_grad(idx, t, grad, ws)):
            with pytest.raises((ValueError, TypeError)):
                f()
    for f in (lambda: gq.gq_embed(idx, Fake((0, 16), F32), out),
              lambda: gq.gq_embed_grad(idx, dy, Fake((0, 16), F32), ws),
              lambda: gq.gq_embed_grad(idx, dy, grad, Fake(1 << 20, F32)),
              lambda: gq.gq_embed_grad(idx, dy, grad, None)):
        with pytest.raises((ValueError, TypeError, AttributeError)):
            f()
