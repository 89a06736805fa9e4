"""nt_paged_tree_attn in fp32 with NaNs of every payload in keys and queries:
the rows whose scores they are in are NaN, no others."""
import numpy as np
import pytest
import torch

from test_gpu_drafts import F32, check, make_case, nt  # noqa: F401
from test_gpu_drafts_edges import KERNELS, MIXED, NARROW, WIDE, at, by

pytestmark = pytest.mark.gpu

# the payload in the lowest bits, in those that a 19-bit part keeps, and in all
PATTERNS = [0x7f800001, 0xff800001, 0x7f801fff, 0x7f802000, 0x7fc00000, 0xffffffff]


def put(t, index, pattern):
    """A bit pattern in place of an element (an assignment of a float may quiet the NaN)."""
    t.view(torch.int32)[index] = int(np.uint32(pattern).view(np.int32))


@pytest.mark.parametrize("shape", [MIXED, WIDE, NARROW])
@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("kernel", KERNELS)
def test_keys(nt, kernel, pattern, shape):
    """One key of the context, and one drafted token's that some see."""
    b = max(i for i, (x, n) in enumerate(zip(shape["ctx"], shape["ns"])) if x > 4 and n)
    other = max(i for i, n in enumerate(shape["ns"]) if n > 4 and i != b)

    def edit(kp, vp, table, q, bits):
        for s, x, h, c in ((b, 3, 0, 2), (other, shape["ctx"][other] + 2, -1, 9)):
            page, row = at(shape, table, s, x)
            put(kp, (page, h, row, c), pattern)

    c = make_case(**shape, dtype=F32, seed=21, edit=edit)
    assert int(torch.isnan(c["kp"]).sum()) == 2
    got = by(nt, c, kernel)
    if got:
        # (check() compares the log-sum-exp where the plain one is a number)
        check(c, got[0], None)
        nan = torch.isnan(got[0].cpu()).all(2)
        assert torch.equal(torch.isnan(got[1].cpu()), nan.T)
        assert bool(nan[sum(shape["ns"][:b]):sum(shape["ns"][:b + 1]), :shape["H"] // shape["Hk"]].all())


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("kernel", KERNELS)
def test_queries(nt, kernel, pattern):
    def edit(kp, vp, table, q, bits):
        put(q, (5, 3, 7), pattern)

    c = make_case(**MIXED, dtype=F32, seed=22, edit=edit)
    got = by(nt, c, kernel)
    if got:
        check(c, got[0], None)
        nan = torch.isnan(got[0].cpu())
        assert bool(nan[5, 3].all()) and int(nan.sum()) == 64 and bool(torch.isnan(got[1][3, 5]))
        assert int(torch.isnan(got[1]).sum()) == 1
