"""The library's C-ABI files on a HIP runtime of the host
(tests/host_runtime/runtime.cpp), in which a chosen call fails: what a failed
allocation or copy leaves behind, and refusals that need a live handle."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from gradient_compression_allreduce_amd.build import CSRC
from tests.conftest import ROOT

GQ_OK, GQ_ERR_INVALID, GQ_ERR_HIP = 0, 1, 4
GOOD = 0x10000


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ is not available")
    out = str(tmp_path_factory.mktemp("host") / "libhost.so")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run(
        [cxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-D__HIP_PLATFORM_AMD__",
         "-I", os.path.join(rocm, "include"), "-o", out,
         os.path.join(ROOT, "tests", "host_runtime", "runtime.cpp"),
         os.path.join(CSRC, "gq_abi.cpp"), os.path.join(CSRC, "gq_tensors.cpp")],
        check=True, capture_output=True, text=True, timeout=300)
    # (launchers that no test reaches are looked for when they are called)
    L = ctypes.CDLL(out, mode=os.RTLD_LAZY)
    vp, f32, i64 = ctypes.c_void_p, ctypes.c_float, ctypes.c_int64
    L.gq_last_error.restype = ctypes.c_char_p
    L.gq_units_create.argtypes = [vp, i64, vp]
    L.gq_units_destroy.argtypes = [vp]
    L.gq_pipe_create.argtypes = [vp, i64, vp, i64, ctypes.c_int32, vp]
    L.gq_pipe_destroy.argtypes = [vp]
    L.gq_tensors_create.argtypes = [vp, vp, vp, i64, vp]
    L.gq_tensors_destroy.argtypes = [vp]
    L.gq_tensors_info.argtypes = [vp, vp, vp, vp]
    L.gq_tensors_norm.argtypes = [vp, f32, vp, vp, vp]
    L.gq_tensors_clip.argtypes = [vp, vp, f32, f32, f32, vp, vp]
    return L


def _list(lib, at, numel, dt=None):
    """(status, handle) of a list of tensors at these addresses."""
    x, n = np.array(at, np.uint64), np.array(numel, np.int64)
    t = np.array(dt if dt is not None else [0] * len(at), np.int32)
    h = ctypes.c_void_p()
    st = lib.gq_tensors_create(x.ctypes.data, n.ctypes.data, t.ctypes.data, len(at), ctypes.byref(h))
    return st, h


def test_failed_list_leaves_no_error(lib):
    """Whichever runtime call of gq_tensors_create fails: no memory stays
    allocated, and no error is left for the thread's next call to report."""
    at, numel = [GOOD, GOOD + (1 << 20)], [100, 5000]
    st, good = _list(lib, at, numel)
    assert st == GQ_OK
    live, before = lib.host_live(), lib.host_calls()
    st, h = _list(lib, at, numel)
    n_calls = lib.host_calls() - before
    assert st == GQ_OK and lib.gq_tensors_destroy(h) == GQ_OK and n_calls >= 6
    for k in range(1, n_calls + 1):
        lib.host_fail_in(k)
        st, h = _list(lib, at, numel)
        assert st == GQ_ERR_HIP and not h.value, k
        assert b"out of memory" in lib.gq_last_error(), k
        assert lib.host_live() == live, k
        assert lib.hipPeekAtLastError() == 0, k
        assert lib.gq_tensors_norm(good, 1.0, 1 << 30, None, None) == GQ_OK, k
    lib.host_fail_in(0)
    assert lib.gq_tensors_destroy(good) == GQ_OK


def _units(lib):
    off = np.array([0, 5, 70_000, 70_001, 400_000], np.int64)
    h = ctypes.c_void_p()
    return lib.gq_units_create(off.ctypes.data, 4, ctypes.byref(h)), h


def _pipe(lib):
    off = np.array([0, 5, 70_000, 70_001, 400_000], np.int64)
    buckets = np.array([0, 2, 4], np.int64)
    h = ctypes.c_void_p()
    return lib.gq_pipe_create(off.ctypes.data, 4, buckets.ctypes.data, 2, 0, ctypes.byref(h)), h


@pytest.mark.parametrize("make,destroy", [(_units, "gq_units_destroy"), (_pipe, "gq_pipe_destroy")])
def test_failed_tables_leave_no_error(lib, make, destroy):
    """The same of gq_units_create and gq_pipe_create."""
    live, before = lib.host_live(), lib.host_calls()
    st, h = make(lib)
    n_calls = lib.host_calls() - before
    assert st == GQ_OK and getattr(lib, destroy)(h) == GQ_OK
    assert lib.host_live() == live and n_calls > 10
    for k in range(1, n_calls + 1):
        lib.host_fail_in(k)
        st, h = make(lib)
        assert st == GQ_ERR_HIP and not h.value, k
        assert lib.host_live() == live, k
        assert lib.hipPeekAtLastError() == 0, k
    lib.host_fail_in(0)


def test_failed_pipe_keeps_its_error_text(lib):
    """A bucket's table that cannot be made: gq_pipe_create tells why."""
    before = lib.host_calls()
    st, h = _pipe(lib)
    n_calls = lib.host_calls() - before
    assert st == GQ_OK and lib.gq_pipe_destroy(h) == GQ_OK
    for k in range(1, n_calls + 1):
        lib.host_fail_in(k)
        st, h = _pipe(lib)
        assert st == GQ_ERR_HIP and b"out of memory" in lib.gq_last_error(), (k, lib.gq_last_error())
    lib.host_fail_in(0)


MiB = 1 << 20


def test_norm_inside_a_list(lib):
    """A norm or norms that lie in a tensor of the list would be read and
    written, or written twice, by the call: refused, at every place of the tensors and with
    the smallest overlap; the places between and beside them are accepted."""
    # fp32 at 1 MiB, bf16 at 2 MiB (odd length), an empty one, fp32 at 3 MiB
    at, numel, dt = [3 * MiB, MiB, 0, 2 * MiB], [5000, 100, 0, 9], [0, 0, 1, 2]
    st, t = _list(lib, at, numel, dt)
    assert st == GQ_OK
    spans = [(MiB, MiB + 400), (2 * MiB, 2 * MiB + 18), (3 * MiB, 3 * MiB + 20_000)]
    far = 64 * MiB
    inside, outside = [], []
    for b, e in spans:
        inside += [b, b + 4, (e - 1) & ~3]
        outside += [b - 4, (e + 3) & ~3]
    for p in inside:
        before = lib.host_launches()
        for call in (lambda: lib.gq_tensors_norm(t, 1.0, p, None, None),
                     lambda: lib.gq_tensors_norm(t, 1.0, far, p, None),
                     lambda: lib.gq_tensors_norm(t, 1.0, far, p - 12, None),
                     lambda: lib.gq_tensors_clip(t, p, 1.0, 0.0, 1.0, None, None),
                     lambda: lib.gq_tensors_clip(t, p, 1.0, 0.0, 1.0, t, None)):
            assert call() == GQ_ERR_INVALID, hex(p)
            assert b"lies in a tensor" in lib.gq_last_error(), lib.gq_last_error()
        assert lib.host_launches() == before
    # norms around the whole of a tensor
    assert lib.gq_tensors_norm(t, 1.0, far, 2 * MiB - 4, None) == GQ_ERR_INVALID
    for p in outside:
        assert lib.gq_tensors_norm(t, 1.0, p, None, None) == GQ_OK, hex(p)
        assert lib.gq_tensors_clip(t, p, 1.0, 0.0, 1.0, None, None) == GQ_OK, hex(p)
    for b, e in spans:
        assert lib.gq_tensors_norm(t, 1.0, far, b - 16, None) == GQ_OK
        assert lib.gq_tensors_norm(t, 1.0, far, (e + 3) & ~3, None) == GQ_OK
    # one of the norms as the norm
    for k in range(4):
        assert lib.gq_tensors_norm(t, 1.0, far + 4 * k, far, None) == GQ_ERR_INVALID, k
        assert b"norms" in lib.gq_last_error()
    for p in (far - 4, far + 16):
        assert lib.gq_tensors_norm(t, 1.0, p, far, None) == GQ_OK
    # into another list: that one's tensors are written, the list's own are only read
    st, out = _list(lib, [a and a + 8 * MiB for a in at], numel, dt)
    assert st == GQ_OK
    for p in inside:
        assert lib.gq_tensors_clip(t, p, 1.0, 0.0, 1.0, out, None) == GQ_OK, hex(p)
        assert lib.gq_tensors_clip(t, p + 8 * MiB, 1.0, 0.0, 1.0, out, None) == GQ_ERR_INVALID
        assert b"lies in a tensor" in lib.gq_last_error()
    # a list without elements has no place that could be taken
    st, none = _list(lib, [0, 0], [0, 0])
    assert st == GQ_OK and lib.gq_tensors_norm(none, 1.0, far, far + 4, None) == GQ_OK
    assert lib.gq_tensors_clip(none, far, 1.0, 0.0, 1.0, None, None) == GQ_OK
    for h in (t, out, none):
        assert lib.gq_tensors_destroy(h) == GQ_OK


def test_memory_of_a_list(lib):
    """What a list allocates is what the header says."""
    with open(os.path.join(ROOT, "include", "gq.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    assert ("24 bytes for each started 4096 elements of a tensor, 24 for each tensor that is "
            "empty or longer than 4096, and 4104 more") in text
    for numel in ([1], [0], [4096], [4097], [8193], [0, 0, 5], [4097] * 300, [1, 70_000, 0, 4096]):
        at = [MiB * (k + 1) for k in range(len(numel))]
        st, h = _list(lib, at, numel)
        n, count, size = (ctypes.c_int64() for _ in range(3))
        assert st == GQ_OK
        assert lib.gq_tensors_info(h, *(ctypes.byref(v) for v in (n, count, size))) == GQ_OK
        tiles = sum(-(-m // 4096) for m in numel)
        more = sum(m == 0 or m > 4096 for m in numel)
        assert (n.value, count.value) == (sum(numel), len(numel))
        assert size.value == 24 * tiles + 24 * more + 4104, numel
        assert lib.gq_tensors_destroy(h) == GQ_OK
