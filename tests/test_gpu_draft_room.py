"""A drafted step over DevicePagedCache that runs out of pages, or of room for
tokens, eager and captured: lengths, table, stack and the pages' contents stay
as they were, and the steps after it are as if it had not been."""
import pytest
import torch

from test_gpu_drafts import BF, DEV, _i32, nt  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured,side", [(False, False), (False, True), (True, False)])
def test_room_runs_out(nt, captured, side):
    """``side``: on a stream given by argument."""
    from variable_length_batching_gb300.paged import DevicePagedCache
    B, T, page, d, n_pages = 3, 24, 4, 64, 9
    cache = DevicePagedCache(B, 12, n_pages, page, 1, d, BF)
    k, v, q = (torch.zeros(T, h, d, dtype=BF, device=DEV) for h in (1, 1, 2))
    counts, parents = _i32([0] * B), torch.full((T,), -1, dtype=torch.int32, device=DEV)
    kept, cu_kept, n_kept = _i32([0] * T), _i32([0] * (B + 1)), _i32([0] * B)
    torch.cuda.synchronize()
    other = torch.cuda.Stream() if side else None

    def step():
        with torch.cuda.stream(other):
            grown = cache.lengths + counts
        cu, pos0, slots, lacking = cache.resize(grown, T, stream=other)
        bits, _ = nt.nt_draft_tree(parents, cu, 16, pos0, stream=other)
        cache.write(k, v, slots, stream=other)
        cache.attend_tree(q, cu, 16, bits, stream=other)
        cache.keep(kept, cu_kept, pos0, stream=other, lacking=lacking)
        with torch.cuda.stream(other):
            after = pos0 + n_kept
        cache.resize(after, stream=other, lacking=lacking)
        return lacking

    run = step
    if captured:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            result = step()

        def run():
            graph.replay()
            return result

    at = [[] for _ in range(B)]                          # what each row's positions hold

    def state():
        torch.cuda.synchronize()
        n = int(cache.n_free)
        return [x.cpu().clone() for x in (cache.lengths, cache.block_table, cache.n_free, cache.free_pages[:n])] + [
            x.cpu().view(torch.int16).clone() for x in (cache.pages.k, cache.pages.v)]

    def held(b):
        table = cache.block_table[b].tolist()
        return [float(cache.pages.k[table[x // page], 0, x % page, 5]) for x in range(len(at[b]))]

    value = 0
    for ns, paths, good in [([5, 2, 3], [[1, 3], [0], []], True),
                            ([9, 9, 9], [[2, 4], [1], [0]], False),         # 27 tokens in room for 24
                            ([12, 2, 2], [[0, 5], [1], [1]], True),
                            ([8, 8, 8], [[1, 2], [1], [3]], True),
                            ([4, 15, 1], [[3], [2, 7, 8, 9, 10, 14], [0]], True),
                            ([16, 4, 4], [[1, 2, 3], [2], [1, 3]], False),  # pages
                            ([2, 1, 1], [[1], [0], [0]], True)]:
        tokens = torch.arange(value, value + T, dtype=torch.float32) % 200 + 1
        value += 37
        for x in (k, v):
            x.copy_(tokens.to(BF)[:, None, None].expand_as(x))
        counts.copy_(_i32(ns)), n_kept.copy_(_i32([len(p) for p in paths]))
        flat = sum(paths, [])
        kept[:len(flat)] = _i32(flat)
        cu_kept[1:] = _i32([len(p) for p in paths]).cumsum(0)
        before = state()
        lacking = run()
        after = state()
        nt.nt_device_status()
        assert (not any(lacking.tolist())) == good
        if not good:
            assert all(torch.equal(x, y) for x, y in zip(before, after))
            continue
        first = 0
        for b in range(B):
            at[b] += [float(tokens[first + i]) for i in paths[b]]
            first += ns[b]
        assert cache.lengths.tolist() == [len(x) for x in at]
        assert [held(b) for b in range(B)] == at
