"""Drafted steps as they are used: room made, masks and positions, keys and
values written, attended to, the accepted ones kept; with the table on the host
and on the device, eager and captured, against a plain model of the cache."""
import random

import numpy as np
import pytest
import torch

from _drafts import bits_of, random_parents, tree_attn, tree_bound
from test_gpu_drafts import BF, DEV, F32, _i32, nt  # noqa: F401

pytestmark = pytest.mark.gpu


class Model:
    """Keys and values of each sequence, (length, H_kv, d)."""

    def __init__(self, rows, Hk, d, dtype):
        self.k = [torch.zeros(0, Hk, d, dtype=dtype) for _ in range(rows)]
        self.v = [torch.zeros(0, Hk, d, dtype=dtype) for _ in range(rows)]
        self.dtype = dtype

    def extend(self, rows, ns, k, v):
        at = 0
        for b, n in zip(rows, ns):
            self.k[b] = torch.cat([self.k[b], k[at:at + n]])
            self.v[b] = torch.cat([self.v[b], v[at:at + n]])
            at += n

    def keep(self, rows, ns, kept):
        for b, n, ks in zip(rows, ns, kept):
            first = self.k[b].shape[0] - n
            at = list(range(first)) + [first + x for x in ks]
            self.k[b], self.v[b] = self.k[b][at], self.v[b][at]

    def check(self, rows, ns, q, bits, o):
        """o against the model's attention of the packed tokens."""
        lens = [self.k[b].shape[0] for b in rows]
        page = max(lens + [1])
        pool = [torch.zeros(len(rows), x[0].shape[1], page, x[0].shape[2], dtype=self.dtype) for x in (self.k, self.v)]
        for i, b in enumerate(rows):
            pool[0][i, :, :lens[i]], pool[1][i, :, :lens[i]] = self.k[b].transpose(0, 1), self.v[b].transpose(0, 1)
        table = torch.arange(len(rows), dtype=torch.int32)[:, None]
        ro, _, mag, cond = tree_attn(pool[0], pool[1], q, ns, table, lens, bits)
        err = (o.double().cpu() - ro).abs()
        assert bool((err <= tree_bound(ro, mag, cond, page, self.dtype)).all())


def a_path(parents, r):
    """The tokens from a root down: an accepted branch."""
    path, at = [], -1
    while True:
        below = [i for i, p in enumerate(parents) if p == at]
        if not below or r.random() < 0.2:
            return path
        at = r.choice(below)
        path.append(at)


@pytest.mark.parametrize("dtype,page,H,Hk,d", [(BF, 16, 8, 2, 64), (BF, 24, 4, 4, 128), (F32, 5, 4, 2, 32)])
def test_host_table(nt, dtype, page, H, Hk, d):
    from variable_length_batching_gb300.paged import PagedCache
    r, rng = random.Random(d), np.random.default_rng(d)
    mk = lambda n, h: torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).to(dtype)
    cache, model = PagedCache(200, page, Hk, d, dtype), Model(5, Hk, d, dtype)
    seqs = [cache.add() for _ in range(5)]

    def step(rows, ns, parents):
        s = cache.step([seqs[b] for b in rows], ns)
        q, k, v = mk(s.tokens, H), mk(s.tokens, Hk), mk(s.tokens, Hk)
        cache.write(s, k.to(DEV), v.to(DEV))
        before = [model.k[b].shape[0] for b in rows]
        model.extend(rows, ns, k, v)
        bits = None
        if parents:
            flat = _i32([p for ps in parents for p in ps])
            bits, pos = nt.nt_draft_tree(flat, s.cu_seqlens, s.max_new, s.pos0)
            want, depths = bits_of(parents, s.max_new)
            assert torch.equal(bits.cpu(), want)
            assert pos.tolist() == [x + p for x, ds in zip(before, depths) for p in ds]
        o = cache.attend_tree(s, q.to(DEV), bits)
        model.check(rows, ns, q, None if bits is None else bits.cpu(), o)
        return s

    step([0, 1, 2], [70, 3, 120], None)                       # prompts
    step([0, 3], [33, 1], None)                               # a further piece
    for n in range(4):
        rows = r.sample(range(5), 4)
        ns = [r.randint(1, 40) for _ in rows]
        parents = [random_parents(m, rng) for m in ns]
        s = step(rows, ns, parents)
        kept = [a_path(p, r) for p in parents]
        cache.keep(s, kept)
        model.keep(rows, ns, kept)
    for b in range(5):
        assert cache.table.length[seqs[b]] == model.k[b].shape[0]
    full = [b for b in range(5) if model.k[b].shape[0]]
    fork = cache.fork(seqs[full[0]])
    s = cache.step([fork], [3])
    k, v = mk(3, Hk), mk(3, Hk)
    cache.write(s, k.to(DEV), v.to(DEV))
    cache.keep(s, [[2]])                                      # in the fork's own copy
    s = step(full, [1] * len(full), None)
    q = mk(len(full), H)
    nt.nt_device_status()
    model.check(full, [1] * len(full), q, None, cache.attend(s, q.to(DEV)))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,page,H,Hk,d", [(BF, 16, 8, 2, 64), (F32, 7, 4, 2, 64)])
def test_device_table(nt, dtype, page, H, Hk, d, captured):
    """The same with the table on the device; captured, one graph is replayed
    for every step, with other counts, trees and accepted tokens."""
    from variable_length_batching_gb300.paged import DevicePagedCache
    r, rng = random.Random(page), np.random.default_rng(page)
    B, T, max_new = 6, 150, 40
    cache, model = DevicePagedCache(B, 40, 150, page, Hk, d, dtype), Model(B, Hk, d, dtype)
    mk = lambda h: torch.from_numpy(rng.standard_normal((T, h, d)).astype(np.float32)).to(dtype)
    q, k, v = (torch.zeros(T, h, d, dtype=dtype, device=DEV) for h in (H, Hk, Hk))
    counts, parents = _i32([0] * B), torch.full((T,), -1, dtype=torch.int32, device=DEV)
    kept, cu_kept, n_kept = _i32([0] * T), _i32([0] * (B + 1)), _i32([0] * B)

    def step():
        cu, pos0, slots, lacking = cache.resize(cache.lengths + counts, T)
        bits, positions = nt.nt_draft_tree(parents, cu, max_new, pos0)
        cache.write(k, v, slots)
        o = cache.attend_tree(q, cu, max_new, bits)
        cache.keep(kept, cu_kept, pos0)
        cache.resize(pos0 + n_kept)
        return o, positions, lacking, bits

    run = step
    if captured:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            results = step()

        def run():
            graph.replay()
            return results

    for n in range(8):
        ns = [r.choice([0, 1, 1, r.randint(1, 20), r.randint(1, max_new)]) for _ in range(B)]
        while sum(ns) > T:
            ns[ns.index(max(ns))] = 1
        trees = [random_parents(m, rng) for m in ns]
        paths = [a_path(p, r) for p in trees]
        hq, hk, hv = mk(H), mk(Hk), mk(Hk)
        q.copy_(hq), k.copy_(hk), v.copy_(hv)
        counts.copy_(_i32(ns)), n_kept.copy_(_i32([len(p) for p in paths]))
        N = sum(ns)
        parents.fill_(-1), kept.fill_(0)
        parents[:N] = _i32([p for t in trees for p in t])
        kept[:sum(map(len, paths))] = _i32([x for p in paths for x in p])
        cu_kept.copy_(_i32(np.concatenate([[0], np.cumsum([len(p) for p in paths])]).tolist()))
        o, positions, lacking, bits = run()
        assert lacking.tolist() == [0, 0]
        nt.nt_device_status()
        before = [x.shape[0] for x in model.k]
        model.extend(range(B), ns, hk, hv)
        want, depths = bits_of(trees, max_new)
        assert torch.equal(bits[:N].cpu(), want)
        assert positions[:N].tolist() == [x + p for x, ds in zip(before, depths) for p in ds]
        model.check(range(B), ns, hq[:N], want, o[:N])
        model.keep(range(B), ns, paths)
        assert cache.lengths.tolist() == [x.shape[0] for x in model.k]
    # the pages in use and the free ones are all of them
    used = cache.block_table[cache.block_table >= 0].tolist() + cache.free_pages[:int(cache.n_free)].tolist()
    assert sorted(used) == list(range(150))
    # one token per row, and more than there are pages
    before = cache.lengths.tolist()
    ones = [1] * B
    cu, pos0, slots, lacking = cache.resize(cache.lengths + 1, B)
    hq, hk, hv = mk(H)[:B], mk(Hk)[:B], mk(Hk)[:B]
    cache.write(hk.to(DEV), hv.to(DEV), slots)
    model.extend(range(B), ones, hk, hv)
    model.check(range(B), ones, hq, None, cache.attend(hq.to(DEV)))
    lacking = cache.resize(torch.full_like(cache.lengths, 40 * page), 40 * page * B)[3]
    assert int(lacking[0]) > 0 and cache.lengths.tolist() == [x + 1 for x in before]
    nt.nt_device_status()
