"""The page table's host logic, without a GPU: sequences extended, forked,
freed and compacted at random, against a model that keeps every sequence's
tokens and moves page contents as the copy lists say."""
import random

import pytest

from variable_length_batching_gb300.paged import OutOfPages, PageTable


def _check(t: PageTable):
    """Every page is free once, or held by as many sequences as its count."""
    held = {}
    for s, pages in t.pages.items():
        assert len(pages) == -(-t.length[s] // t.page_size) and len(set(pages)) == len(pages)
        for p in pages:
            held[p] = held.get(p, 0) + 1
    assert t.refs == [held.get(p, 0) for p in range(t.n_pages)]
    assert sorted(t.free_pages) == [p for p in range(t.n_pages) if p not in held]


@pytest.mark.parametrize("page_size", [1, 3, 16])
@pytest.mark.parametrize("seed", range(8))
def test_random_use_keeps_every_token(seed, page_size):
    r = random.Random(seed)
    t = PageTable(40, page_size)
    pool = [[None] * page_size for _ in range(40)]       # what the pages hold
    want = {}                                            # what each sequence should read
    token = 0

    def apply(copies):
        srcs, dsts = [a for a, _ in copies], [b for _, b in copies]
        assert len(set(dsts)) == len(dsts) and not set(srcs) & set(dsts)
        for a, b in copies:
            pool[b] = list(pool[a])

    for _ in range(400):
        what = r.choice(["add", "extend", "extend", "extend", "fork", "free", "compact"])
        live = sorted(want)
        if what == "add":
            want[t.add()] = []
        elif what == "extend" and live:
            seqs = r.sample(live, r.randint(1, len(live)))
            counts = [r.choice([0, 1, 1, r.randint(0, 3 * page_size)]) for _ in seqs]
            before = (list(t.refs), {s: list(p) for s, p in t.pages.items()}, dict(t.length), sorted(t.free_pages))
            try:
                apply(t.extend(seqs, counts))
            except OutOfPages:
                assert before == (t.refs, t.pages, t.length, sorted(t.free_pages))
                continue
            for s, n in zip(seqs, counts):
                for _ in range(n):
                    x = len(want[s])
                    pool[t.pages[s][x // page_size]][x % page_size] = token
                    want[s].append(token)
                    token += 1
        elif what == "fork" and live:
            s = r.choice(live)
            want[t.fork(s)] = list(want[s])
        elif what == "free" and live:
            s = r.choice(live)
            t.free(s)
            del want[s]
        elif what == "compact":
            apply(t.compact())
            used = sum(x > 0 for x in t.refs)
            assert all(x > 0 for x in t.refs[:used])
        _check(t)
        for s, toks in want.items():
            assert [pool[t.pages[s][x // page_size]][x % page_size] for x in range(len(toks))] == toks


def test_all_sharers_extend_at_once():
    """Three sequences on one partly filled page extend together: two get
    copies, the last keeps the page."""
    t = PageTable(4, 4)
    a = t.add()
    t.extend([a], [2])
    b, c = t.fork(a), t.fork(a)
    copies = t.extend([a, b, c], [1, 1, 1])
    assert len(copies) == 2 and len({t.pages[s][0] for s in (a, b, c)}) == 3
    _check(t)


def test_full_last_page_stays_shared():
    t = PageTable(4, 4)
    a = t.add()
    t.extend([a], [4])
    b = t.fork(a)
    assert t.extend([b], [1]) == []
    assert t.pages[a][0] == t.pages[b][0] and len(t.pages[b]) == 2
    _check(t)


def test_refusals():
    t = PageTable(2, 4)
    a = t.add()
    with pytest.raises(KeyError):
        t.extend([a + 1], [1])
    with pytest.raises(KeyError):
        t.free(a + 1)
    with pytest.raises(KeyError):
        t.fork(a + 1)
    with pytest.raises(ValueError):
        t.extend([a, a], [1, 1])
    with pytest.raises(ValueError):
        t.extend([a], [-1])
    with pytest.raises(ValueError):
        t.extend([a], [1, 2])
    with pytest.raises(OutOfPages):
        t.extend([a], [9])
    with pytest.raises(ValueError):
        PageTable(-1, 4)
    with pytest.raises(ValueError):
        PageTable(4, 0)
    t.free(a)
    with pytest.raises(KeyError):
        t.free(a)
