"""Slot maps of tables with a page below 0 where a row has positions: no slot
of it may be the -1 that stands for a token without a place."""
import pytest
import torch

from test_gpu_drafts import DEV, _i32, nt  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,have,bad", [(1, 0, -1), (1, 2, -1), (4, 3, -1), (4, 2, -1), (4, 0, -1), (16, 15, -1), (4, 3, -7),
                                           (1, 0, -2 ** 31)])
@pytest.mark.parametrize("rows", [1, 3, 700])
def test_pages_below_0(nt, rows, page, have, bad):
    """A page in the table (where the row's last one is not full) or on the
    stack, in the middle row: its tokens' slots are -2, flagged, not written."""
    b, grown = rows // 2, page + 2
    held = -(-have // page)                                 # pages of a row before, and after
    wide = -(-(have + grown) // page)
    table = torch.full((rows, wide), -1, dtype=torch.int32)
    table[:, :held] = torch.arange(rows * held, dtype=torch.int32).view(rows, held)
    used = rows * wide
    free = torch.arange(used - 1, rows * held - 1, -1, dtype=torch.int32)
    full = have % page == 0
    at = (held if full else held - 1)                       # the bad page's column
    if full:
        free[len(free) - 1 - b * (wide - held)] = bad       # of rank b (wide - held) among the taken ones
    else:
        table[b, at] = bad
    want = []
    final = table.clone()
    final[:, held:] = free.flip(0).view(rows, wide - held)
    for r in range(rows):
        for x in range(have, have + grown):
            p = int(final[r, x // page])
            want.append(-2 if p < 0 else p * page + x % page)
    assert -2 in want and -1 not in want
    table, stack = table.to(DEV), torch.cat((free, torch.full((rows * held,), -1, dtype=torch.int32))).to(DEV)
    lengths = _i32([have] * rows)
    cu, pos0, slots, lacking = nt.nt_paged_resize(table, lengths, stack, _i32([len(free)]), page, lengths + grown,
                                                  rows * grown + 3)
    with pytest.raises(nt.NTError) as e:
        nt.nt_device_status()
    assert e.value.status == 6 and lacking.tolist() == [0, 0]
    assert slots.tolist() == want + [-1] * 3 and torch.equal(table.cpu(), final)
    pages = nt.KVPages(*(torch.zeros(used, 1, page, 8, device=DEV) for _ in range(2)))
    kv = torch.ones(len(slots), 1, 8, device=DEV)
    nt.nt_paged_write_slots(pages, kv, kv, slots)
    with pytest.raises(nt.NTError) as e:
        nt.nt_device_status()
    written = torch.zeros(used * page)
    written[[s for s in want if s >= 0]] = 1
    for pool in (pages.k, pages.v):
        assert torch.equal(pool[:, 0, :, 3].flatten().cpu(), written)
