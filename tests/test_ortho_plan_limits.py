"""Limits of gq_ortho_create, without a GPU: a plan beyond them is refused
before tables of its size are built."""
import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT

SIDES = ((1 << 15, 1 << 22), (1 << 22, 1 << 15), (1 << 15, 1 << 19))

CHILD = """
import ctypes, sys
import numpy as np
from gradient_compression_allreduce_amd import gq

def peak():     # KiB, of this program alone
    return int(open("/proc/self/status").read().split("VmHWM:")[1].split()[0])

rows, cols = int(sys.argv[1]), int(sys.argv[2])
gq.gq_mx4_sizes(1, 1)
before = peak()
a = [np.array([v], np.int64) for v in (0, rows, cols)]
h = ctypes.c_void_p()
st = gq.lib.gq_ortho_create(*(v.ctypes.data for v in a), 1, 5, None, 1e-7, None, ctypes.byref(h))
after = peak()
print(st, after - before, gq.gq_last_error())
"""


@pytest.mark.parametrize("rows,cols", SIDES)
def test_too_many_elements(rows, cols):
    """Sides within their limits, 2^34 elements or more together: refused, with
    the number of elements in the message, and with far less host memory than
    the 24 bytes per 4096 elements of the tile table it would need (100 MB at
    the limit)."""
    env = dict(os.environ, PYTHONPATH=ROOT)
    out = subprocess.run([sys.executable, "-c", CHILD, str(rows), str(cols)], env=env, cwd=ROOT,
                         capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    status, kib, text = out.stdout.strip().split(" ", 2)
    assert int(status) == 1, out.stdout       # GQ_ERR_INVALID
    assert text.startswith("gq_ortho_create") and "2^34" in text
    assert int(kib) < 30 * 1024, out.stdout


def test_header_states_the_limit():
    with open(os.path.join(ROOT, "include", "gq.h")) as f:
        text = f.read()
    doc = text[text.index("gq_ortho_create --"):text.index("gq_status gq_ortho_create(")]
    assert "2^34" in doc


def test_tiles_of_no_plan():
    from gradient_compression_allreduce_amd import gq
    assert gq.lib.gq_ortho_tiles(None, None, None) == gq.GQ_ERR_INVALID
    assert gq.gq_last_error().startswith("gq_ortho_tiles")
