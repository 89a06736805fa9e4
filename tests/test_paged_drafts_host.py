"""PagedCache's drafted steps without a GPU: what is refused, what the device
is asked to move, and what the table is left with."""
import contextlib

import pytest
import torch

from variable_length_batching_gb300 import paged


class Pages:
    device = torch.device("cpu")


@pytest.fixture
def cache(monkeypatch):
    c = object.__new__(paged.PagedCache)
    c.table, c.pages, c.moved, c.fail, c.capturing = paged.PageTable(12, 4), Pages(), [], False, False

    def keep(pages, kept, cu, table, pos0, stream=None):
        if c.fail:
            raise RuntimeError("launch failed")
        c.moved.append((kept.tolist(), cu.tolist(), pos0.tolist()))

    monkeypatch.setattr(paged.nt, "nt_paged_keep", keep)
    monkeypatch.setattr(paged.nt, "nt_paged_copy", lambda *a, **kw: None)
    monkeypatch.setattr(torch.Tensor, "pin_memory", lambda t: t)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: c.capturing)
    return c


def _state(t):
    return list(t.refs), list(t.free_pages), {s: list(p) for s, p in t.pages.items()}, dict(t.length)


def test_keep(cache):
    a, b, e = cache.add(), cache.add(), cache.add()
    cache.step([a, b, e], [6, 4, 0])
    step = cache.step([b, a, e], [7, 3, 2])
    cache.keep(step, [[0, 3, 5], [2], []])
    assert cache.moved == [([0, 3, 5, 2], [0, 3, 4, 4], [4, 6, 0])]
    assert cache.table.length == {a: 7, b: 7, e: 0}
    assert [len(cache.table.pages[s]) for s in (a, b, e)] == [2, 2, 0]
    assert sorted(cache.table.free_pages + cache.table.pages[a] + cache.table.pages[b]) == list(range(12))


def test_nothing_to_move(cache):
    """The first tokens of a step kept: nothing is launched."""
    a, b = cache.add(), cache.add()
    step = cache.step([a, b], [5, 6])
    cache.keep(step, [[0, 1], list(range(6))])
    assert cache.moved == [] and cache.table.length == {a: 2, b: 6}


@pytest.mark.parametrize("kept", [[[0]], [[0], [1], [2]], [[0, 0], []], [[2, 1], []], [[-1], []], [[3], []], [[], [2]]])
def test_refused(cache, kept):
    a, b = cache.add(), cache.add()
    step = cache.step([a, b], [3, 2])
    before = _state(cache.table)
    with pytest.raises(ValueError):
        cache.keep(step, kept)
    assert _state(cache.table) == before and cache.moved == []


def test_only_the_last_step(cache):
    a, b = cache.add(), cache.add()
    old = cache.step([a, b], [3, 2])
    cache.step([a], [1])
    before = _state(cache.table)
    with pytest.raises(ValueError, match="changed"):
        cache.keep(old, [[1], [1]])
    gone = cache.step([b], [1])
    cache.free(b)
    with pytest.raises(KeyError):
        cache.keep(gone, [[0]])
    assert before[3][a] == cache.table.length[a] and cache.moved == []


def test_forked_since(cache):
    """A fork shares the step's pages: nothing is moved in them, but what
    stays in place may be kept."""
    a = cache.add()
    step = cache.step([a], [6])
    f = cache.fork(a)
    before = _state(cache.table)
    with pytest.raises(ValueError, match="forked"):
        cache.keep(step, [[0, 2]])
    assert _state(cache.table) == before and cache.moved == []
    cache.keep(step, [[0, 1, 2]])
    assert cache.table.length == {a: 3, f: 6} and len(cache.table.pages[f]) == 2 and len(cache.table.pages[a]) == 1


def test_compacted_since(cache):
    """The step's block table names the old places."""
    a, b = cache.add(), cache.add()
    cache.step([a, b], [5, 5])
    step = cache.step([b], [3])
    cache.free(a)
    cache.compact()
    before = _state(cache.table)
    with pytest.raises(ValueError, match="moved"):
        cache.keep(step, [[1]])
    assert _state(cache.table) == before and cache.moved == []


def test_a_move_that_fails_gives_nothing_up(cache):
    a = cache.add()
    step = cache.step([a], [6])
    before = _state(cache.table)
    cache.fail = True
    with pytest.raises(RuntimeError):
        cache.keep(step, [[2]])
    cache.fail, cache.capturing = False, True
    with pytest.raises(RuntimeError, match="capture"):
        cache.keep(step, [[2]])
    assert _state(cache.table) == before


def test_shorten():
    t = paged.PageTable(6, 4)
    a, b = t.add(), t.add()
    t.extend([a, b], [9, 4])
    for seqs, lengths in [([a], [10]), ([a], [-1]), ([a, a], [1, 1]), ([a], [1, 2])]:
        with pytest.raises(ValueError):
            t.shorten(seqs, lengths)
    t.shorten([a, b], [4, 0])
    assert len(t.pages[a]) == 1 and t.pages[b] == [] and len(t.free_pages) == 5


def test_queries_are_the_whole_step(cache):
    a = cache.add()
    step = cache.step([a], [6])
    with pytest.raises(ValueError, match="6 new tokens"):
        cache.attend_tree(step, torch.zeros(5, 2, 32))
