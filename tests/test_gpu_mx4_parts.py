"""gq_mx4_product with K in parts, on tiles of every size: exact values, each
output type, running sums, row strides, and NaN scales of every part."""
import pytest
import torch

from tests import mx4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# m, n, tile that splits K, lengths: the last part whole, short, of an odd
# number of groups, and ending inside a group or a block
CASES = [(3900, 1020, 256, (15009, 15872, 16384)), (8000, 1000, 256, (8192, 7700, 7181)),
         (3001, 1500, 256, (6001, 6700, 11008)), (1000, 1000, 128, (12000, 16384, 13313)),
         (300, 500, 64, (12289, 14000, 16384))]


@pytest.fixture(scope="module")
def gq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from gradient_compression_allreduce_amd import gq as mod
    return mod


def _parts_of(m, n, k, tile):
    """Parts of K that a tile of this size takes where it splits K: up to as
    many as give each of 256 compute units a work group, of an even number of
    groups of 512 elements."""
    groups = -(-k // 512)
    want = min(256 // (-(-m // tile) * -(-n // tile)), groups // 2)
    if want < 2:
        return 1
    per = (-(-groups // want) + 1) // 2 * 2
    return -(-groups // per)


def _parts(gq, m, n, k, tile):
    """Parts of K, by the workspace, which no other tile would take."""
    parts = gq.gq_mx4_product_workspace(m, n, k) // (4 * m * n)
    assert parts >= 2 and [t for t in (64, 128, 256) if _parts_of(m, n, k, t) == parts] == [tile]
    return parts


def _operand(gen, rows, k):
    """Codes with zeros behind the row's end, and scales 126 and 127."""
    nb = ref.blocks(k)
    q = torch.randint(0, 256, (rows, nb * 16), dtype=torch.uint8, device="cuda", generator=gen)
    left = k - 32 * (nb - 1)
    last = q[:, (nb - 1) * 16:]
    last[:, (left + 1) // 2:] = 0
    if left % 2:
        last[:, left // 2] &= 15
    s = torch.randint(126, 128, (rows, nb), dtype=torch.uint8, device="cuda", generator=gen)
    return q.view(-1), s


@pytest.mark.parametrize("m,n,tile,ks", CASES)
def test_exact(gq, m, n, tile, ks):
    """Terms are multiples of 2^-4 of at most 36, and 16384 of them and a C of
    whole numbers below 2^8 stay below 2^20, so binary32 sums are exact in any
    order, and the output is one rounding of them."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    for k in ks:
        parts = _parts(gq, m, n, k, tile)
        qa, sa = _operand(gen, m, k)
        qb, sb = _operand(gen, n, k)
        a, b = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
        gq.gq_mx4_reduce_dequant([qa], [sa.view(-1)], m, k, a.view(-1))
        gq.gq_mx4_reduce_dequant([qb], [sb.view(-1)], n, k, b.view(-1))
        p = torch.mm(a, b.t().contiguous())
        ws = torch.full((gq.gq_mx4_product_workspace(m, n, k),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        for dt, add, gap, offset in (("f32", False, 0, 0), ("f32", True, 3, 1), ("bf16", False, 0, 0),
                                     ("f16", False, 4, 3)):
            say("parts", parts, "tile", tile, m, n, k, dt, "add", add, "gap", gap)
            flat = torch.full((offset + m * (n + gap),), -7.0, dtype=TORCH[dt], device="cuda")
            c = flat[offset:].view(m, n + gap)[:, :n]
            if add:
                c.copy_(torch.randint(-255, 256, (m, n), device="cuda", generator=gen).float())
            want = flat.clone()
            wc = want[offset:].view(m, n + gap)[:, :n]
            wc.copy_(((wc if add else 0) + p).to(TORCH[dt]))
            gq.gq_mx4_product(qa, sa.view(-1), qb, sb.view(-1), k, c, accumulate=add, workspace=ws)
            assert torch.equal(flat, want), (m, n, k, dt, add)


@pytest.mark.parametrize("m,n,tile,ks", CASES)
def test_nan_scales(gq, m, n, tile, ks):
    """A NaN scale in any part reaches its own row or column and nothing else."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    k = ks[0]
    parts, nb = _parts(gq, m, n, k, tile), ref.blocks(k)
    qa, sa = _operand(gen, m, k)
    qb, sb = _operand(gen, n, k)
    rows, cols = [], []
    for p in range(parts + 1):
        at = min(nb - 1, p * nb // parts)
        rows.append((37 * p + 5) % m)
        cols.append((71 * p + 11) % n)
        sa[rows[-1], at] = 255
        sb[cols[-1], at] = 255
    sa[m - 1, nb - 1] = sb[n - 1, nb - 1] = 255
    say("nan", m, n, k, "parts", parts)
    c = torch.zeros(m, n, device="cuda")
    ws = torch.empty(gq.gq_mx4_product_workspace(m, n, k), dtype=torch.uint8, device="cuda")
    gq.gq_mx4_product(qa, sa.view(-1), qb, sb.view(-1), k, c, workspace=ws)
    want = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    want[rows + [m - 1], :] = True
    want[:, cols + [n - 1]] = True
    assert torch.equal(torch.isnan(c), want)
