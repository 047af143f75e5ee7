"""The binding's lazily filled tables under two first calls at once, without a
GPU: while one thread is half way through filling a table, another must not
see half of it."""
import sys
import threading

import pytest
import torch


@pytest.fixture()
def gq():
    from gradient_compression_allreduce_amd import gq as mod
    return mod


class Slow:
    """A module whose attribute `name` holds up the first thread that asks for
    it until another thread has gone through."""

    def __init__(self, real, name, replace):
        self._real, self._name, self._replace = real, name, replace
        self.waiting, self.go = threading.Event(), threading.Event()

    def __getattr__(self, name):
        if name == self._name and not self.waiting.is_set():
            self.waiting.set()
            assert self.go.wait(30)
        if name in self._replace:
            return self._replace[name]
        return getattr(self._real, name)


def _two_calls(slow, call):
    """What `call` gives in a thread held up by `slow`, and in another one that
    runs meanwhile."""
    got = {}

    def run(key):
        try:
            got[key] = call()
        except Exception as e:       # shown by the caller
            got[key] = e

    first = threading.Thread(target=run, args=("first",))
    first.start()
    try:
        assert slow.waiting.wait(30)
        run("second")
    finally:
        slow.go.set()
        first.join(30)
    return got["first"], got["second"]


def test_stream_lookup(gq, monkeypatch):
    slow = Slow(torch._C, "_cuda_getDevice", {"_cuda_getDevice": lambda: 3,
                                              "_cuda_getCurrentRawStream": lambda dev: 100 + dev})
    monkeypatch.setattr(gq, "_RAW", type(gq._RAW)())
    monkeypatch.setattr(torch, "_C", slow)
    assert _two_calls(slow, gq._raw_stream) == (103, 103)


def test_dtype_table(gq, monkeypatch):
    slow = Slow(torch, "bfloat16", {})
    monkeypatch.setattr(gq, "_TORCH", {})
    monkeypatch.setitem(sys.modules, "torch", slow)
    first, second = _two_calls(slow, lambda: sorted(gq._dt()))
    assert first == second and "code" in first
