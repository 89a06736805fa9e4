"""Attention of drafted tokens over a paged cache (nt_paged_tree_attn) on the
GPU against a 64-bit plain form."""
import math

import numpy as np
import pytest
import torch

from _drafts import bits_of, make_pool, random_parents, tree_attn, tree_bound

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def nt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_batching_gb300 import build, nt as ntmod
    build.build()
    return ntmod


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cu(ns):
    return _i32(np.concatenate([[0], np.cumsum(ns)]).tolist())


def make_case(ctx, ns, page, H, Hk, d, dtype, kind="tree", seed=0, max_new=None, edit=None):
    rng = np.random.default_rng(seed + 50)
    lens = [c + n for c, n in zip(ctx, ns)]
    kp, vp, table = make_pool(lens, page, Hk, d, dtype, seed)
    q = (2 * torch.from_numpy(rng.standard_normal((sum(ns), H, d)).astype(np.float32))).to(dtype)
    max_new = max(list(ns) + [1]) if max_new is None else max_new
    bits = None if kind == "causal" else bits_of([random_parents(n, rng, kind) for n in ns], max_new)[0]
    if edit:
        edit(kp, vp, table, q, bits)
    return dict(kp=kp, vp=vp, table=table, q=q, bits=bits, ns=list(ns), lens=lens, max_new=max_new, dtype=dtype)


def call(nt, c, scale=None, want_lse=True, **kw):
    pages = nt.KVPages(c["kp"].to(DEV), c["vp"].to(DEV))
    bits = None if c["bits"] is None else c["bits"].to(DEV)
    o, lse = nt.nt_paged_tree_attn(pages, c["q"].to(DEV), _cu(c["ns"]), c["table"].to(DEV), _i32(c["lens"]),
                                   c["max_new"], bits=bits, scale=scale, want_lse=want_lse, **kw)
    nt.nt_device_status()
    return o, lse


def call_kernel(nt, c, kernel, scale=None, cluster=0):
    """The same by a kernel by name; None where it does not take the call."""
    pages = nt.KVPages(c["kp"].to(DEV), c["vp"].to(DEV))
    bits = None if c["bits"] is None else c["bits"].to(DEV)
    try:
        got = nt.nt_selftest_paged_tree_attn(kernel, pages, c["q"].to(DEV), _cu(c["ns"]), c["table"].to(DEV),
                                             _i32(c["lens"]), c["max_new"], bits=bits, scale=scale, cluster=cluster)
    except nt.NTError as e:
        assert e.status == 2 and kernel
        return None
    nt.nt_device_status()
    return got


def check(c, o, lse, scale=None):
    ro, rl, mag, cond = tree_attn(c["kp"], c["vp"], c["q"], c["ns"], c["table"], c["lens"], c["bits"], scale)
    n = max(c["lens"] + [0])
    got = o.double().cpu()
    fine = torch.isfinite(ro)
    assert torch.equal(torch.isnan(got), torch.isnan(ro))
    odd = ~fine & ~torch.isnan(ro)
    assert torch.equal(got[odd], ro[odd])
    err = (got - ro).abs()[fine]
    bound = tree_bound(ro, mag, cond, n, c["dtype"])[fine]
    assert bool((err <= bound).all()), float((err / bound).max())
    if c["dtype"] == F32 and err.numel():
        assert float(err.max()) <= 1e-5 * max(float(ro[fine].abs().max()), 1e-30)
    if lse is not None:
        got = lse.double().cpu()
        none = torch.isinf(rl) & (rl < 0)
        assert torch.equal(torch.isinf(got) & (got < 0), none)
        lb = (32 * cond[..., 0].T + 64 + n / 4 + 4 * rl.abs()) * 2.0 ** -24
        assert bool(((got - rl).abs() <= lb)[~none].all())


SHAPES = [  # contexts, new tokens, page, H, Hk, d
    ([0], [1], 16, 1, 1, 64),
    ([777], [8], 16, 12, 12, 64),
    ([0], [5], 16, 2, 1, 64),
    ([0, 5, 100, 63, 64, 65, 1, 130, 16, 0], [3, 0, 7, 1, 64, 2, 0, 33, 16, 1], 16, 8, 2, 64),
    ([63, 127, 128, 129, 15], [1, 1, 64, 65, 17], 16, 8, 1, 128),
    ([300, 7, 0, 1000], [4, 4, 4, 4], 8, 4, 4, 128),
    ([300, 7, 0, 1000], [9, 30, 41, 2], 24, 14, 2, 128),      # 7 heads to a key head, pages of 24
    ([300, 41], [12, 40], 1, 2, 2, 32),
    ([513, 2], [20, 3], 7, 6, 2, 64),
    ([100, 700], [60, 3], 48, 32, 2, 64),                     # 16 heads to a key head
    ([100, 700], [256, 130], 256, 24, 1, 128),                # 24, and the largest trees
    ([50, 3], [100, 7], 128, 40, 1, 64),
    ([2500], [33], 64, 8, 1, 128),                            # one long sequence over many CTAs
    ([0] * 150 + [1] * 150, [1] * 300, 16, 2, 1, 64),         # more sequences than threads of a CTA
    ([3000, 1, 1, 2000, 5], [3, 200, 1, 70, 9], 100, 5, 5, 32),
    ([200, 31], [3, 2], 32, 80, 1, 64),                       # 80 heads to a key head
    ([90, 500], [1, 2], 16, 300, 2, 32),                      # 150
]


@pytest.mark.parametrize("kind", ["tree", "causal"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_tree_attn(nt, shape, dtype, kind):
    ctx, ns, page, H, Hk, d = SHAPES[shape]
    c = make_case(ctx, ns, page, H, Hk, d, dtype, kind, seed=shape)
    check(c, *call(nt, c))
    takes = {0: True, 1: dtype == BF and d > 32 and page % 8 == 0 and H // Hk <= 128,
             2: dtype == BF and d < 128 and page % 8 == 0, 3: True}
    for kernel in (0, 1, 2, 3):
        got = call_kernel(nt, c, kernel)
        assert (got is not None) == takes[kernel]
        if got:
            check(c, *got)
