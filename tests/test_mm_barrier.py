"""The barrier of the matrix-core tile loops (csrc/gq_mm.h), by its compiled
form: a buffer in LDS is loaded again after a barrier behind its last reads, so
each wave has to wait for its reads before it passes, wherever the compiler
puts the matrix instructions that use them."""
import os
import re
import subprocess

import pytest

from gradient_compression_allreduce_amd import build

KERNEL = """
#include "%s"
using namespace gq;
extern "C" __global__ __launch_bounds__(256) void tiles(const void *p, const void *q, float *out,
                                                        int groups, int i0) {
    using S = MmSmall;
    MM_LDS(S);
    const MmRows a = mm_rows(p, 4096, 0, 64, 64), b = mm_rows(q, 4096, 0, 64, 64);
    MmAcc<S> acc = {};
    // something under a branch between the barrier and the reads
    auto extra = [&](MmAcc<S> &c, const char *lds, int step, int) {
        if (step == i0) c.c[0][0][0][0] += *reinterpret_cast<const float *>(lds);
    };
    mm_loop<S, false>(a, b, MmScale{}, 0, groups, mm_lds, nullptr, extra, acc);
    reinterpret_cast<mm_f32x4 *>(out)[threadIdx.x] = acc.c[0][0][0] + acc.c[0][1][1];
}
"""


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    d = tmp_path_factory.mktemp("mm")
    src = d / "tiles.hip"
    src.write_text(KERNEL % os.path.join(build.CSRC, "gq_mm.h"))
    out = d / "tiles.s"
    subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "-S", "--offload-device-only", str(src),
                    "-o", str(out)], check=True, capture_output=True, timeout=300)
    return out.read_text()


def test_reads_are_waited_for_at_every_barrier(listing):
    lines = [s.strip() for s in listing.splitlines()]
    at = [i for i, s in enumerate(lines) if re.match(r"s_barrier\b", s)]
    assert len(at) >= 3       # two in the loop, one behind it
    asm, forced = False, []
    for i, s in enumerate(lines):
        if s.startswith(";;#ASM"):
            asm = "START" in s
        elif asm and re.match(r"s_waitcnt\b.*lgkmcnt\(0\)", s):
            forced.append(i)
    loop = 0
    for i in at:
        # back to what is waited for, in a block of inline assembly, so that it
        # does not hang on the compiler's order; no LDS access in between
        j = i - 1
        while j >= 0 and j not in forced and not re.match(r"ds_|\.LBB|s_barrier", lines[j]):
            j -= 1
        loop += j in forced
    assert loop >= 2, "a barrier of the loop does not wait for the wave's LDS reads"
