"""nt_paged_tree_attn with many short items to a CTA: sequences of one key tile
behind such of several, with one and two row tiles, whose new tokens' values
are not finite here and there.  Streams of the tensor-memory kernel that have
nothing to do in an item must not run ahead of those that do."""
import math

import numpy as np
import pytest
import torch

from test_gpu_drafts import BF, DEV, _cu, _i32, call, call_kernel, check, make_case, nt  # noqa: F401

pytestmark = pytest.mark.gpu


def sequences(what, rng):
    """(contexts, new tokens, H, H_kv): 800 items and more, five to each of 152 SMs."""
    B = 100
    if what == "one tile":                        # the first and last rows of a tile, in one row tile
        ns = rng.integers(20, 129, B)
        return [int(rng.integers(0, 129 - n)) for n in ns], ns, 8, 8
    if what == "three and one":                   # odd numbers of key tiles in turn
        ns = rng.integers(20, 61, B)
        return [int(rng.integers(260, 320)) if i % 2 else int(rng.integers(0, 66)) for i in range(B)], ns, 8, 8
    if what == "two row tiles and one":
        ns = np.where(rng.random(B) < 0.4, rng.integers(33, 65, B), rng.integers(1, 33, B))
        ns[0] = 64
        return [int(x) for x in np.where(rng.random(B) < 0.7, rng.integers(0, 60, B), rng.integers(60, 500, B))], ns, 32, 8
    ns = rng.integers(1, 30, B)                   # lengths of every kind
    return [int(x) for x in rng.choice([0, 3, 100, 127, 128, 200, 300, 420, 600], B)], ns, 8, 8


@pytest.mark.parametrize("kind", ["causal", "tree"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["one tile", "three and one", "two row tiles and one", "mixed"])
@pytest.mark.parametrize("seed", range(3))
def test_values_not_finite_in_many_items(nt, seed, what, d, kind):
    """In two of three sequences the first, a middle or the last new token has
    an infinite or NaN value in an early and a late column: the rows that see
    it get it, no other does, and every run gives the same bits."""
    rng = np.random.default_rng(seed)
    ctx, ns, H, Hk = sequences(what, rng)
    ns = [int(n) for n in ns]

    def edit(kp, vp, table, q, bits):
        for b, (c, n) in enumerate(zip(ctx, ns)):
            if b % 3 == 2:
                continue
            for i in {0, n - 1, int(rng.integers(0, n))}:
                x = c + i
                page, row = int(table[b, x // 16]), x % 16
                for col in (int(rng.integers(0, 32)), d - 1 - int(rng.integers(0, 32))):
                    vp[page, int(rng.integers(0, Hk)), row, col] = [math.inf, -math.inf, math.nan][int(rng.integers(0, 3))]

    c = make_case(ctx, ns, 16, H, Hk, d, BF, kind, seed=seed, edit=edit)
    first = call_kernel(nt, c, 1)
    check(c, *first)
    check(c, *call(nt, c))
    pages = nt.KVPages(c["kp"].to(DEV), c["vp"].to(DEV))
    bits = None if c["bits"] is None else c["bits"].to(DEV)
    q, cu, table, lens = c["q"].to(DEV), _cu(ns), c["table"].to(DEV), _i32(c["lens"])
    outs = [torch.zeros_like(q) for _ in range(25)]
    for o in outs:
        nt.nt_selftest_paged_tree_attn(1, pages, q, cu, table, lens, c["max_new"], bits=bits, out=o)
    nt.nt_device_status()
    want = first[0].view(torch.int16)
    assert all(torch.equal(o.view(torch.int16), want) for o in outs)
