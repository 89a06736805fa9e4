"""What a step with drafted tokens needs around its attention, on the GPU
against plain forms: nt_paged_resize, nt_paged_write_slots, nt_draft_tree and
nt_paged_keep."""
import random

import numpy as np
import pytest
import torch

from _drafts import bits_of, make_pool, random_parents

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
    return _i32(np.concatenate([[0], np.cumsum(ns)]).astype(int).tolist())


# ---- tables -----------------------------------------------------------------

class State:
    """A table on the device, and the same as lists."""

    def __init__(self, B, max_pages, n_pages, page, seed=0):
        r = random.Random(seed)
        self.page, self.max_pages = page, max_pages
        self.free = list(range(n_pages))
        r.shuffle(self.free)
        self.n_free = n_pages
        self.rows = [[-1] * max_pages for _ in range(B)]
        self.lens = [0] * B
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
        self.lengths = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.dfree, self.dn = _i32(self.free), _i32([n_pages])

    def resize(self, new, tokens):
        """The plain form: (cu, pos0, slots, lacking)."""
        pages = lambda n: -(-n // self.page)
        old = list(self.lens)
        gone = sum(max(pages(o) - pages(n), 0) for o, n in zip(old, new))
        come = sum(max(pages(n) - pages(o), 0) for o, n in zip(old, new))
        add = sum(max(n - o, 0) for o, n in zip(old, new))
        lacking = [max(0, come - gone - self.n_free), max(0, add - tokens)]
        if any(lacking):
            return [0] * (len(old) + 1), old, [-1] * tokens, lacking
        top = self.n_free + gone - 1
        rank = 0
        for row, o, n in zip(self.rows, old, new):
            for p in range(pages(n), pages(o)):
                self.free[top - rank], row[p] = row[p], -1
                rank += 1
        rank, slots, cu = 0, [], [0]
        for row, o, n in zip(self.rows, old, new):
            for p in range(pages(o), pages(n)):
                row[p] = self.free[top - rank]
                rank += 1
            slots += [row[x // self.page] * self.page + x % self.page for x in range(o, n)]
            cu.append(cu[-1] + max(n - o, 0))
        self.n_free += gone - come
        self.lens = list(new)
        return cu, old, slots + [-1] * (tokens - len(slots)), lacking

    def step(self, nt, new, tokens):
        got = nt.nt_paged_resize(self.table, self.lengths, self.dfree, self.dn, self.page, _i32(new), tokens)
        want = self.resize(new, tokens)
        for g, w in zip(got, want):
            assert g.tolist() == w
        self.same()
        return got

    def same(self):
        assert self.table.tolist() == self.rows
        assert self.lengths.tolist() == self.lens
        assert self.dfree.tolist() == self.free and self.dn.tolist() == [self.n_free]


@pytest.mark.parametrize("B,max_pages,n_pages,page", [(1, 40, 40, 16), (3, 9, 20, 1), (33, 8, 150, 7), (512, 6, 1500, 16),
                                                      (513, 6, 1500, 16), (1700, 5, 4000, 3), (5, 600, 2000, 8)])
def test_resize(nt, B, max_pages, n_pages, page):
    """Rows that grow, shrink, stay, end and begin, several times over; too
    few pages and too little room leave everything as it was."""
    r = random.Random(B)
    s = State(B, max_pages, n_pages, page, seed=B)
    cap = max_pages * page
    lacked = 0
    for step in range(12):
        most = [cap, 1, cap // 2, page + 1, 0, cap][step % 6]
        new = [r.choice([o, min(cap, o + 1), r.randint(0, most), 0 if r.random() < 0.2 else o]) for o in s.lens]
        add = sum(max(n - o, 0) for o, n in zip(s.lens, new))
        tokens = max(0, add + r.choice([0, 0, 5, 100, -1]))
        got = s.step(nt, new, tokens)
        lacked += any(got[3].tolist())
    nt.nt_device_status()
    # and back: table and stack as they were
    before = s.table.clone(), s.dfree.clone(), s.dn.clone()
    old = list(s.lens)
    up = [min(cap, o + 1) for o in old]
    if not any(s.step(nt, up, sum(up) - sum(old))[3].tolist()):
        s.step(nt, old, 0)
        assert all(torch.equal(x, y) for x, y in zip(before, (s.table, s.dfree, s.dn)))


def test_resize_long_row(nt):
    """One row of many pages: they are dealt out over the threads."""
    s = State(2, 5000, 6000, 4, seed=1)
    s.step(nt, [19999, 3], 20002)
    s.step(nt, [1, 17000], 17000)
    s.step(nt, [0, 0], 0)
    assert s.n_free == 6000
    nt.nt_device_status()


def test_resize_lacking(nt):
    s = State(2, 10, 5, 4, seed=2)
    assert s.step(nt, [12, 9], 30)[3].tolist() == [1, 0]       # six pages of five
    assert s.step(nt, [12, 8], 19)[3].tolist() == [0, 1]       # 20 tokens in 19
    assert s.step(nt, [12, 8], 20)[3].tolist() == [0, 0]
    assert s.step(nt, [4, 16], 8)[3].tolist() == [0, 0]        # two pages change hands
    nt.nt_device_status()


def test_resize_flags(nt):
    """Lengths outside the table leave their row; a broken count leaves all."""
    s = State(3, 4, 12, 4, seed=3)
    s.step(nt, [5, 5, 5], 15)
    got = nt.nt_paged_resize(s.table, s.lengths, s.dfree, s.dn, 4, _i32([17, -1, 6]), 4)
    with pytest.raises(nt.NTError) as e:
        nt.nt_device_status()
    assert e.value.status == 6
    want = s.resize([5, 5, 6], 4)
    assert [g.tolist() for g in got] == [list(w) for w in want]
    s.same()
    for bad in (-1, 13, 11):            # 11: with the pages given back, more than there are
        dn = _i32([bad])
        nt.nt_paged_resize(s.table, s.lengths, s.dfree, dn, 4, _i32([0, 0, 0]), 0)
        with pytest.raises(nt.NTError):
            nt.nt_device_status()
        assert dn.tolist() == [bad]
        s.same()


def test_resize_empty(nt):
    t, e = torch.zeros(0, 3, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    cu, pos0, slots, lacking = nt.nt_paged_resize(t, e, _i32([1, 2]), _i32([2]), 4, e, 5)
    nt.nt_device_status()
    assert cu.tolist() == [0] and pos0.numel() == 0 and slots.tolist() == [-1] * 5 and lacking.tolist() == [0, 0]


# ---- write by slots ------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,page,Hk,d", [(1, 16, 1, 64), (9, 16, 8, 128), (700, 7, 2, 40), (5000, 64, 3, 32)])
def test_write_slots(nt, dtype, T, page, Hk, d):
    g = torch.Generator().manual_seed(T)
    pool = -(-2 * T // page) + 1
    kp, vp = (torch.randn(pool, Hk, page, d, generator=g).to(dtype) for _ in range(2))
    k, v = (torch.randn(T, Hk, d, generator=g).to(dtype) for _ in range(2))
    slots = torch.randperm(pool * page, generator=g)[:T]
    slots[::5] = -1
    pages = nt.KVPages(kp.to(DEV), vp.to(DEV))
    fused = torch.cat((k, v), 1).to(DEV)
    nt.nt_paged_write_slots(pages, fused[:, :Hk], fused[:, Hk:], slots.to(DEV))
    nt.nt_device_status()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            kp[s // page, :, s % page], vp[s // page, :, s % page] = k[t], v[t]
    assert torch.equal(pages.k.cpu(), kp) and torch.equal(pages.v.cpu(), vp)


def test_write_slots_flags(nt):
    z, one = torch.zeros(2, 1, 4, 8, device=DEV), torch.ones(3, 1, 8, device=DEV)
    for bad in (8, -2, 1 << 40):
        pages = nt.KVPages(z.clone(), z.clone())
        nt.nt_paged_write_slots(pages, one, one, torch.tensor([0, bad, 7], device=DEV))
        with pytest.raises(nt.NTError) as e:
            nt.nt_device_status()
        assert e.value.status == 6 and int(pages.k.sum()) == 16 and int(pages.v.sum()) == 16


# ---- trees ----------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["tree", "chain", "roots"])
@pytest.mark.parametrize("ns,max_new", [([1], 1), ([64, 0, 5], 64), ([65, 1, 64, 63], 65), ([256, 255, 0, 3, 128, 129], 256),
                                        ([2] * 300, 7), ([0, 0], 4), ([], 4)])
def test_draft_tree(nt, ns, max_new, kind):
    rng = np.random.default_rng(len(ns))
    parents = [random_parents(n, rng, kind) for n in ns]
    bits, depths = bits_of(parents, max_new)
    pos0 = [int(x) for x in rng.integers(0, 1 << 30, len(ns))]
    flat = _i32(sum(parents, []) + [7] * 5)                  # five tokens that only fill up the batch
    if not ns:                                               # tokens with no segments are refused
        with pytest.raises(nt.NTError) as e:
            nt.nt_draft_tree(flat, _cu(ns), max_new, pos0=_i32(pos0))
        assert e.value.status == 1
        flat = flat[:0]
    got, pos = nt.nt_draft_tree(flat, _cu(ns), max_new, pos0=_i32(pos0))
    nt.nt_device_status()
    n = sum(ns)
    assert torch.equal(got.cpu()[:n], bits.view(n, got.shape[1]))
    assert pos.tolist()[:n] == [p + x for p, d in zip(pos0, depths) for x in d]
    if ns:
        assert not got[n:].any() and not pos[n:].any()
        assert nt.nt_draft_tree(flat, _cu(ns), max_new)[1].tolist()[:n] == sum(depths, [])


def test_draft_tree_flags(nt):
    for parents, cu, want in (([-1, 1, 0], [0, 3], [1, 2, 5]),      # a token on itself
                              ([-2, 0, 0], [0, 3], [1, 3, 5]),
                              ([-1, 0, 5], [0, 3], [1, 3, 4]),
                              ([-1, 0, 0], [0, 4], None), ([-1, 0, 0], [-1, 2], None)):
        bits = torch.full((3, 1), -9, dtype=torch.int64, device=DEV)
        nt.nt_draft_tree(_i32(parents), _i32(cu), 3, bits=bits)
        with pytest.raises(nt.NTError) as e:
            nt.nt_device_status()
        assert e.value.status == 6
        if want:
            assert bits.flatten().tolist() == want
    bits = torch.full((5, 1), -9, dtype=torch.int64, device=DEV)
    nt.nt_draft_tree(_i32([-1, 0, 1, -1, 0]), _i32([0, 3, 5]), 2, bits=bits)      # three tokens where two are allowed
    with pytest.raises(nt.NTError):
        nt.nt_device_status()
    assert bits.flatten().tolist() == [-9, -9, -9, 1, 3]


# ---- kept tokens ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page,Hk,d", [(16, 8, 128), (1, 1, 8), (7, 3, 40), (64, 12, 64), (24, 130, 256)])
def test_keep(nt, dtype, page, Hk, d):
    """Paths whose places overlap their sources, none, all, many tokens."""
    r = random.Random(page)
    ctx = [0, 5, 33, 100, 17, 2, 64]
    new = [9, 40, 0, 300, 64, 7, 1]
    kept = [[0, 1, 2], [1, 2, 3, 5, 8, 13, 21, 39], [], list(range(3, 300)), sorted(r.sample(range(64), 30)), list(range(7)),
            [0]]
    kp, vp, table = make_pool([c + n for c, n in zip(ctx, new)], page, Hk, d, dtype, seed=page)
    pages = nt.KVPages(kp.to(DEV), vp.to(DEV))
    nt.nt_paged_keep(pages, _i32(sum(kept, [])), _cu([len(x) for x in kept]), table.to(DEV), _i32(ctx))
    nt.nt_device_status()
    for pool, got in ((kp, pages.k), (vp, pages.v)):
        want = pool.clone()
        for b, path in enumerate(kept):
            for i, k in enumerate(path):
                s, t = ctx[b] + k, ctx[b] + i
                want[table[b, t // page], :, t % page] = pool[table[b, s // page], :, s % page]
        assert torch.equal(got.cpu(), want)


def test_keep_flags(nt):
    """Indices that do not grow, places outside the table, pages outside the
    pool: flagged, and not moved."""
    x = torch.arange(8, device=DEV, dtype=F32).reshape(2, 1, 4, 1).expand(2, 1, 4, 8).contiguous()
    for kept, table, p0, want in (([1, 1], [[0, 1]], 0, [1, 1, 2, 3, 4, 5, 6, 7]),
                                  ([2, 1], [[0, 1]], 0, [2, 1, 2, 3, 4, 5, 6, 7]),
                                  ([-1, 3], [[0, 1]], 0, [0, 3, 2, 3, 4, 5, 6, 7]),
                                  ([3, 8], [[0, 1]], 0, [3, 1, 2, 3, 4, 5, 6, 7]),
                                  ([1, 5], [[0, 2]], 0, [1, 1, 2, 3, 4, 5, 6, 7]),
                                  ([1, 5], [[0, -1]], 0, [1, 1, 2, 3, 4, 5, 6, 7]),
                                  ([1, 2], [[0, 1]], -1, [0, 1, 2, 3, 4, 5, 6, 7])):
        pages = nt.KVPages(x.clone(), x.clone())
        nt.nt_paged_keep(pages, _i32(kept), _i32([0, 2]), _i32(table), _i32([p0]))
        with pytest.raises(nt.NTError) as e:
            nt.nt_device_status()
        assert e.value.status == 6
        assert pages.k[:, 0, :, 0].flatten().tolist() == want and pages.v[:, 0, :, 7].flatten().tolist() == want
    for cu in ([0, 3], [-1, 2], [2, 1]):
        pages = nt.KVPages(x.clone(), x.clone())
        nt.nt_paged_keep(pages, _i32([1, 2]), _i32(cu), _i32([[0, 1]]), _i32([0]))
        with pytest.raises(nt.NTError):
            nt.nt_device_status()
        assert torch.equal(pages.k, x)
