"""DevicePagedCache's documented step where room was lacking, without a GPU:
the library's calls are stood in for by plain ones on host tensors."""
import pytest
import torch

from variable_length_batching_gb300 import paged


class Pages:
    device = torch.device("cpu")


@pytest.fixture
def cache(monkeypatch):
    """Three rows, pages of four; lengths stand for the table."""
    c = object.__new__(paged.DevicePagedCache)
    c.pages, c.page_size, c.room = Pages(), 4, 6
    c.block_table = c.free_pages = c.n_free = None
    c.lengths = torch.tensor([3, 0, 9], dtype=torch.int32)
    c.kept = []

    def resize(table, lengths, free, n_free, page_size, new, tokens=0, stream=None):
        assert new.dtype == torch.int32 and new.shape == lengths.shape
        old = lengths.clone()
        pages = lambda x: int(((x + 3) // 4).sum())
        gained = (new - old).clamp(min=0)
        lacking = torch.tensor([max(0, pages(new) - c.room), max(0, int(gained.sum()) - tokens)], dtype=torch.int32)
        if lacking.any():
            return torch.zeros(4, dtype=torch.int32), old, torch.full((tokens,), -1), lacking
        lengths.copy_(new)
        return torch.cat((old[:1] * 0, gained.cumsum(0).int())), old, None, lacking

    def keep(pages, kept, cu_kept, table, pos0, stream=None):
        assert cu_kept.dtype == torch.int32 and cu_kept.is_contiguous() and cu_kept.numel() == 4
        for b in range(3):
            c.kept += [(b, int(pos0[b]) + k) for k in kept[cu_kept[b]:cu_kept[b + 1]].tolist()]

    monkeypatch.setattr(paged.nt, "nt_paged_resize", resize)
    monkeypatch.setattr(paged.nt, "nt_paged_keep", keep)
    return c


def step(c, counts, tokens, n_kept):
    """Of each row the tokens 1, 2, ... of the step are kept."""
    ints = lambda x: torch.tensor(x, dtype=torch.int32)
    cu_kept = torch.cat((ints([0]), ints(n_kept).cumsum(0).int()))
    kept = ints([i + 1 for n in n_kept for i in range(n)])
    cu, pos0, slots, lacking = c.resize(c.lengths + ints(counts), tokens)
    c.keep(kept, cu_kept, pos0, lacking=lacking)
    c.resize(pos0 + ints(n_kept), lacking=lacking)
    return lacking.tolist()


def test_a_step_that_has_room(cache):
    assert step(cache, [4, 2, 3], 9, [2, 1, 0]) == [0, 0]
    assert cache.lengths.tolist() == [5, 1, 9] and cache.kept == [(0, 4), (0, 5), (1, 1)]


@pytest.mark.parametrize("counts,tokens", [([30, 2, 3], 40), ([4, 2, 3], 8)])
def test_a_step_that_lacks_room(cache, counts, tokens):
    """Nothing is kept, and no row grows by positions that were never written."""
    assert any(step(cache, counts, tokens, [2, 1, 1]))
    assert cache.lengths.tolist() == [3, 0, 9] and cache.kept == []
    assert step(cache, [4, 2, 3], 9, [1, 0, 1]) == [0, 0]
    assert cache.lengths.tolist() == [4, 0, 10] and cache.kept == [(0, 4), (2, 10)]
