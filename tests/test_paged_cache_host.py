"""PagedCache's own logic, without a GPU: the device calls and streams are
stood in for, and fail where a test wants them to."""
import contextlib
import random

import pytest
import torch

from variable_length_batching_gb300 import paged


class Pages:
    device = torch.device("cpu")


@pytest.fixture
def cache(monkeypatch):
    """Eight pages of four positions; ``cache.copied`` collects the page
    copies, ``cache.fail`` names the call that is to fail."""
    c = object.__new__(paged.PagedCache)
    c.table, c.pages, c.copied, c.fail = paged.PageTable(8, 4), Pages(), [], None
    c.capturing = False

    def copy(pages, src, dst, stream=None):
        if c.fail == "copy":
            raise RuntimeError("launch failed")
        c.copied += list(zip(src.tolist(), dst.tolist()))

    def pin(t):
        if c.fail == "pin":
            raise RuntimeError("no memory")
        return t

    monkeypatch.setattr(paged.nt, "nt_paged_copy", copy)
    monkeypatch.setattr(torch.Tensor, "pin_memory", pin)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: c.capturing)
    return c


def _state(t):
    return list(t.refs), list(t.free_pages), {s: list(p) for s, p in t.pages.items()}, dict(t.length)


def test_retract_is_extend_taken_back():
    r = random.Random(1)
    t = paged.PageTable(30, 4)
    seqs = [t.add() for _ in range(4)]
    t.extend(seqs, [9, 1, 0, 16])
    for _ in range(300):
        if r.random() < 0.3 and len(seqs) < 8:
            seqs.append(t.fork(r.choice(seqs)))
        elif r.random() < 0.2 and len(seqs) > 2:
            t.free(seqs.pop(r.randrange(len(seqs))))
        some = r.sample(seqs, r.randint(1, len(seqs)))
        counts = [r.choice([0, 1, 1, 5, 9]) for _ in some]
        before = _state(t)
        try:
            copies = t.extend(some, counts)
        except paged.OutOfPages:
            t.free(seqs.pop())
            seqs.append(t.add())
            continue
        after = _state(t)
        t.retract(some, counts, copies)
        assert _state(t) == before
        assert t.extend(some, counts) == copies and _state(t) == after
        if r.random() < 0.5:
            t.retract(some, counts, copies)


@pytest.mark.parametrize("what", ["copy", "pin"])
def test_a_step_that_fails_makes_no_room(cache, what):
    a = cache.add()
    cache.step([a], [6])
    b = cache.fork(a)
    before = _state(cache.table)
    cache.fail = what
    with pytest.raises(RuntimeError):
        cache.step([b, a], [3, 1])
    assert _state(cache.table) == before
    cache.fail = None
    step = cache.step([b, a], [3, 1])
    assert step.lengths.tolist() == [9, 7] and step.pos0.tolist() == [6, 6] and step.cu_seqlens.tolist() == [0, 3, 4]
    assert len(cache.copied) == (2 if what == "pin" else 1)


def test_a_compaction_that_fails_moves_nothing(cache):
    a, b = cache.add(), cache.add()
    cache.step([a, b], [9, 9])
    cache.free(a)
    before = _state(cache.table)
    cache.fail = "copy"
    with pytest.raises(RuntimeError):
        cache.compact()
    assert _state(cache.table) == before
    cache.fail = None
    cache.compact()
    assert len(cache.copied) == 3 and sorted(cache.table.pages[b]) == [0, 1, 2]


def test_neither_is_captured(cache):
    """What changes the table now and the pages at a replay is refused."""
    a, b = cache.add(), cache.add()
    cache.step([a, b], [9, 9])
    cache.free(a)
    before = _state(cache.table)
    cache.capturing = True
    for call in (cache.compact, lambda: cache.step([b], [1])):
        with pytest.raises(RuntimeError, match="capture"):
            call()
    assert _state(cache.table) == before and cache.copied == []


def test_a_write_is_the_whole_step(cache, monkeypatch):
    """Fewer tokens than the step made room for would leave positions that
    are attended to and were never written."""
    written = []
    monkeypatch.setattr(paged.nt, "nt_paged_write", lambda pages, k, v, *a, **kw: written.append(k.shape[0]))
    a, b = cache.add(), cache.add()
    step = cache.step([a, b], [5, 2])
    kv = lambda n: torch.zeros(n, 1, 8)
    for n in (0, 6, 8):
        with pytest.raises(ValueError, match="7 new tokens"):
            cache.write(step, kv(n), kv(n))
    cache.write(step, kv(7), kv(7))
    assert written == [7]
