"""Steps that PagedCache.keep refuses although the sequence's length is what
they left it at, without a GPU."""
import random

import pytest
import torch

from test_paged_drafts_host import _state, cache  # noqa: F401
from variable_length_batching_gb300 import paged


def refused(c, step, kept):
    before, moved = _state(c.table), list(c.moved)
    with pytest.raises(ValueError, match="changed"):
        c.keep(step, kept)
    assert _state(c.table) == before and c.moved == moved


def test_after_a_copied_page(cache):  # noqa: F811
    """The step after a fork copies the shared page; its tokens given up, the
    length is the first step's, but the page in its table is the fork's."""
    a = cache.add()
    cache.step([a], [8])
    first = cache.step([a], [3])
    cache.fork(a)
    second = cache.step([a], [1])
    assert first.block_table.tolist() == [[0, 1, 2]] and cache.table.pages[a] == [0, 1, 3]
    cache.keep(second, [[]])
    assert cache.table.length[a] == 11
    refused(cache, first, [[0, 2]])


def test_kept_before(cache):  # noqa: F811
    """A second keep of a step would write over the tokens of the one after it."""
    a = cache.add()
    first = cache.step([a], [4])
    cache.keep(first, [[0, 2]])
    refused(cache, first, [[0]])
    second = cache.step([a], [2])
    refused(cache, first, [[0, 2]])
    cache.keep(second, [[1]])
    assert cache.table.length[a] == 3


def test_pages_that_are_anothers(cache):  # noqa: F811
    """A page of the step is given up and taken by another sequence."""
    a, b = cache.add(), cache.add()
    first = cache.step([a], [8])
    cache.keep(first, [[0]])
    cache.step([b], [4])
    assert cache.table.pages[b] == [1] and first.block_table.tolist() == [[0, 1]]
    cache.step([a], [7])
    assert cache.table.length[a] == 8
    refused(cache, first, [[0, 5]])
    refused(cache, first, [[4, 5]])


def test_still_the_last(cache, monkeypatch):  # noqa: F811
    """What leaves the sequence alone leaves its step the last one: other
    sequences' steps, one of no token, extensions that failed."""
    a, b = cache.add(), cache.add()
    first = cache.step([a], [6])
    cache.step([b, a], [5, 0])
    with pytest.raises(paged.OutOfPages):
        cache.step([a], [100])

    def no_memory(t):
        raise RuntimeError("no memory")

    with monkeypatch.context() as m:                    # the step's room is taken back
        m.setattr(torch.Tensor, "pin_memory", no_memory)
        with pytest.raises(RuntimeError, match="memory"):
            cache.step([a], [3])
    cache.keep(first, [[1, 3]])
    assert cache.moved == [([1, 3], [0, 2], [0])] and cache.table.length == {a: 2, b: 5}


def test_counts_in_the_table():
    """Each cache has its own; a call taken back leaves them as they were."""
    t, u = paged.PageTable(12, 4), paged.PageTable(12, 4)
    a = t.add()
    t.extend([a], [5])
    f = t.fork(a)
    before = dict(t.changes)
    t.retract([f, a], [2, 1], t.extend([f, a], [2, 1]))
    assert t.changes == before == {a: 1, f: 0}
    t.shorten([a], [5])
    assert t.changes[a] == 1
    t.shorten([a], [1])
    t.compact()
    assert t.changes == {a: 2, f: 0} and (t.compactions, u.compactions) == (1, 0)
    t.free(a)
    assert t.changes == {f: 0}


def test_steps_made_by_hand(cache):  # noqa: F811
    """A step without the counts that keep() goes by is refused."""
    a = cache.add()
    s = cache.step([a], [3])
    bare = paged.Step(s.seqs, s.cu_seqlens, s.pos0, s.lengths, s.block_table, s.max_new, s.tokens, s.counts, s.after)
    with pytest.raises(ValueError):
        cache.keep(bare, [[0]])
    assert cache.table.length[a] == 3


@pytest.mark.parametrize("seed", range(12))
def test_random_use(cache, monkeypatch, seed):  # noqa: F811
    """Steps, forks, ends, compactions and keeps of any step so far, against a
    model of every sequence's tokens: a keep is refused, or right."""
    r = random.Random(seed)
    pool = [[None] * 4 for _ in range(12)]
    model, steps, token = {}, [], 0
    kept_some = refused_some = 0

    def move(pages, kept, cu, table, pos0, stream=None):
        kept, cu, table, pos0 = kept.tolist(), cu.tolist(), table.tolist(), pos0.tolist()
        for b in range(len(pos0)):
            for i, k in enumerate(kept[cu[b]:cu[b + 1]]):
                src, dst = pos0[b] + k, pos0[b] + i
                pool[table[b][dst // 4]][dst % 4] = pool[table[b][src // 4]][src % 4]

    def copy(pages, src, dst, stream=None):
        for a, b in zip(src.tolist(), dst.tolist()):
            pool[b] = list(pool[a])

    monkeypatch.setattr(paged.nt, "nt_paged_keep", move)
    monkeypatch.setattr(paged.nt, "nt_paged_copy", copy)
    for _ in range(400):
        what = r.choice(["add", "step", "step", "step", "keep", "keep", "keep", "fork", "free", "compact"])
        live = sorted(model)
        if what == "add" and len(live) < 5:
            model[cache.add()] = []
        elif what == "step" and live:
            seqs = r.sample(live, r.choice([1, 1, 1, min(2, len(live))]))
            counts = [r.choice([0, 1, 2, 2, 3]) for _ in seqs]
            try:
                step = cache.step(seqs, counts)
            except paged.OutOfPages:
                s = r.choice(live)
                cache.free(s)
                del model[s]
                continue
            added = []
            for b, (s, n) in enumerate(zip(seqs, counts)):
                added.append(list(range(token, token + n)))
                for i in range(n):
                    x = int(step.pos0[b]) + i
                    pool[int(step.block_table[b, x // 4])][x % 4] = token
                    model[s] = model[s] + [token]
                    token += 1
            steps.append((step, added))
        elif what == "keep" and steps:
            step, added = r.choice(steps[-r.choice([1, 1, 12]):])
            kept = [sorted(r.sample(range(n), r.randint(0, n))) for n in step.counts]
            before = _state(cache.table)
            try:
                cache.keep(step, kept)
            except (ValueError, KeyError):
                assert _state(cache.table) == before
                refused_some += 1
            else:
                kept_some += 1
                for s, n, new, ks in zip(step.seqs, step.counts, added, kept):
                    first = len(model[s]) - n
                    assert model[s][first:] == new               # the step was the last one
                    model[s] = model[s][:first] + [model[s][first + k] for k in ks]
        elif what == "fork" and live and len(live) < 5:
            s = r.choice(live)
            model[cache.fork(s)] = list(model[s])
        elif what == "free" and live and r.random() < 0.4:
            s = r.choice(live)
            cache.free(s)
            del model[s]
        elif what == "compact" and r.random() < 0.3:
            cache.compact()
        for s, toks in model.items():
            pages = cache.table.pages[s]
            assert cache.table.length[s] == len(toks)
            assert [pool[pages[x // 4]][x % 4] for x in range(len(toks))] == toks
    assert kept_some > 10 and refused_some > 10
