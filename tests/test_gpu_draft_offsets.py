"""nt_draft_tree with a last segment whose offsets do not fit: it is flagged,
and the other segments' masks are as they would be."""
import pytest
import torch

from test_gpu_drafts import DEV, _i32, nt  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu,max_new", [(cu, n) for n in (8, 70, 256) for cu in (
    [0, 4, -1], [0, 8, 4], [0, 4, 9], [0, 8, -2 ** 31], [0, 4, 2 ** 31 - 1])]
    + [([0, 3, 8], 4)])                               # five tokens where four are allowed
def test_last_segment_flagged(nt, cu, max_new):
    n, words = cu[1], -(-max_new // 64)
    for _ in range(20):                               # (CTAs of other segments write at the same time)
        bits = torch.full((8, words), -9, dtype=torch.int64, device=DEV)
        positions = torch.full((8,), -9, dtype=torch.int32, device=DEV)
        nt.nt_draft_tree(_i32([-1, 0, 1, 2, 3, 4, 5, 6]), _i32(cu), max_new, _i32([100, 200]), bits, positions)
        with pytest.raises(nt.NTError) as e:
            nt.nt_device_status()
        assert e.value.status == 6
        assert bits[:, 0].tolist() == [2 ** (i + 1) - 1 for i in range(n)] + [-9] * (8 - n)
        assert bool((bits[:n, 1:] == 0).all()) and bool((bits[n:] == -9).all())
        assert positions.tolist() == [100 + i for i in range(n)] + [-9] * (8 - n)


def test_tokens_behind_a_good_last_segment(nt):
    """An earlier segment is flagged, the tokens behind the last one are filled."""
    bits, positions = (torch.full(s, -9, dtype=t, device=DEV) for s, t in (((8, 1), torch.int64), ((8,), torch.int32)))
    nt.nt_draft_tree(_i32([-1] * 8), _i32([-1, 3, 5]), 4, _i32([10, 20]), bits, positions)
    with pytest.raises(nt.NTError):
        nt.nt_device_status()
    assert bits.flatten().tolist() == [-9] * 3 + [1, 2] + [0] * 3
    assert positions.tolist() == [-9] * 3 + [20] * 2 + [0] * 3


@pytest.mark.parametrize("counts", [[0, 0, 0], [0], []])
def test_step_without_new_tokens(nt, counts):
    """The documented calls of a drafted step, with no token in any sequence."""
    from variable_length_batching_gb300.paged import PagedCache
    cache = PagedCache(8, 4, 2, 64)
    seqs = [cache.add() for _ in counts]
    cache.step(seqs, [3] * len(seqs))
    step = cache.step(seqs, counts)
    parents, kv = _i32([]), torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    bits, positions = nt.nt_draft_tree(parents, step.cu_seqlens, step.max_new, step.pos0)
    cache.write(step, kv, kv)
    o = cache.attend_tree(step, torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV), bits)
    cache.keep(step, [[] for _ in counts])
    nt.nt_device_status()
    assert o.shape == (0, 4, 64) and bits.numel() == 0 and positions.numel() == 0
    assert all(cache.table.length[s] == 3 for s in seqs)
