"""How near paged attention in bf16 comes to fp64: the output's own rounding
and fp32 arithmetic, no more.

A probability reaches the product as the sum of two bf16.  The upper one is
the largest below it, so the rest is at most one step, 2^-7 of it, and is
rounded by half a step, 2^-8 of itself: 2^-15 of each probability."""
import math

import pytest
import torch

from _attn_path import HALF_STEP, U32, paged_attn
from test_gpu_paged import SHAPES, SHORT, _attn_case, nt  # noqa: F401

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("wide", [0, 200000])
@pytest.mark.parametrize("shape", SHAPES + SHORT)
def test_probabilities_keep_their_bits(nt, shape, wide):  # noqa: F811
    lens, page, H, Hk, d = shape
    inputs, o, _ = _attn_case(nt, lens, page, H, Hk, d, BF, seed=11, wide=wide // page)
    kp, vp, table, q = inputs
    ro, _, mag, cond = paged_attn(kp, vp, q, table, lens)
    steps = 2 * 16 * cond + 8 * 2 + max(lens) / 8 + 64           # of fp32, as in attn_bound
    bound = HALF_STEP[BF] * ro.abs() * 1.001 + (2.0 ** -15 + steps * U32) * mag + 1e-38
    err = (o.double().cpu() - ro).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("page,wide", [(16, 0), (16, 200000), (12, 0)])
def test_infinite_values_stay_infinite(nt, page, wide):  # noqa: F811
    """An infinity among the attended values makes its column's outputs that
    infinity, as its product with any probability is, and no other's."""
    n, d = 50, 64

    def edit(kp, vp, table, q):
        vp[table[0, 3 // page], :, 3 % page, 5] = math.inf
        vp[table[0, 40 // page], :, 40 % page, 9] = -math.inf
        kp[:] = 0                                                # all probabilities equal, and exact in bf16
        q[:] = 0

    inputs, o, lse = _attn_case(nt, [n], page, 4, 2, d, BF, edit=edit, wide=wide // page)
    o = o.cpu()
    assert bool((o[:, :, 5] == math.inf).all()) and bool((o[:, :, 9] == -math.inf).all())
    rest = torch.ones(d, dtype=torch.bool)
    rest[[5, 9]] = False
    assert bool(torch.isfinite(o[:, :, rest]).all())
