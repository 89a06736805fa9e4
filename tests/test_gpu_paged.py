"""The paged key/value cache on the GPU: nt_paged_write, nt_paged_copy and
nt_paged_attn against 64-bit plain forms."""
import math

import pytest
import torch

from _attn_path import HALF_STEP, attn_bound, make_pool, paged_attn

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


def _rand(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cu(segs):
    return _i32([0] + torch.tensor(segs).cumsum(0).tolist() if segs else [0])


# ---- write ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("segs,starts,page,Hk,d", [
    ([1], [0], 16, 1, 64),
    ([1] * 9, [0, 15, 16, 17, 31, 5, 100, 63, 64], 16, 8, 128),
    ([5, 0, 1, 130, 0, 64], None, 64, 12, 64),
    ([33, 7, 50], [3, 70, 0], 24, 3, 32),
    ([40, 9], [1, 2], 1, 2, 8),
    ([300], [4], 7, 2, 40),
])
def test_write(nt, dtype, segs, starts, page, Hk, d):
    st = [0] * len(segs) if starts is None else starts
    kp, vp, table = make_pool([s + n for s, n in zip(st, segs)], page, Hk, d, dtype, seed=1)
    T = sum(segs)
    k, v = _rand(2, T, Hk, d, dtype=dtype), _rand(3, T, Hk, d, dtype=dtype)
    pages = nt.KVPages(kp.to(DEV), vp.to(DEV))
    fused = torch.cat((k, v), 1).to(DEV)              # read as slices of one projection
    nt.nt_paged_write(pages, fused[:, :Hk], fused[:, Hk:], _cu(segs), table.to(DEV),
                      pos0=None if starts is None else _i32(starts))
    nt.nt_device_status()
    t = 0
    for b, n in enumerate(segs):
        for i in range(n):
            x = st[b] + i
            kp[table[b, x // page], :, x % page] = k[t]
            vp[table[b, x // page], :, x % page] = v[t]
            t += 1
    assert torch.equal(pages.k.cpu(), kp) and torch.equal(pages.v.cpu(), vp)


def test_write_flags_what_it_cannot_place(nt):
    """Offsets short of T, a position beyond the table, a page outside the
    pool: flagged, nothing written for those tokens."""
    z = torch.zeros(4, 1, 4, 8, device=DEV)
    one = torch.ones(6, 1, 8, device=DEV)
    table = _i32([[0, 9], [-1, 1]])
    for cu, p0, written in (([0, 6, 6], [0, 0], 4),        # page 9 of 4
                            ([0, 0, 6], [0, 0], 2),        # page -1, then page 1
                            ([0, 2, 3], [2, 6], 3),        # three tokens behind cu's end
                            ([0, 1, 6], [-1, 6], 2)):      # position -1; beyond max_pages
        pages = nt.KVPages(z.clone(), z.clone())
        nt.nt_paged_write(pages, one, one, _i32(cu), table, pos0=_i32(p0))
        with pytest.raises(nt.NTError) as ei:
            nt.nt_device_status()
        assert ei.value.status == 6
        assert int(pages.k.sum()) == 8 * written and int(pages.v.sum()) == 8 * written


# ---- copy -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,pool,page,Hk,d", [(1, 2, 16, 1, 64), (448, 900, 1, 2, 8), (449, 900, 8, 1, 32),
                                              (4100, 8200, 1, 1, 16), (5, 11, 24, 3, 128), (3, 7, 100, 12, 128)])
def test_copy(nt, dtype, n, pool, page, Hk, d):
    k, v = _rand(1, pool, Hk, page, d, dtype=dtype).to(DEV), _rand(2, pool, Hk, page, d, dtype=dtype).to(DEV)
    ids = torch.randperm(pool, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    src, dst = ids[:n].contiguous(), ids[n:2 * n].contiguous()
    if n > 2:
        src[1] = src[0]                      # one page to two places
    wk, wv = k.clone(), v.clone()
    wk[dst.long().to(DEV)] = k[src.long().to(DEV)]
    wv[dst.long().to(DEV)] = v[src.long().to(DEV)]
    nt.nt_paged_copy(nt.KVPages(k, v), src, dst)
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_captured_copy_keeps_its_list(nt):
    k = torch.arange(6, device=DEV, dtype=F32).reshape(6, 1, 1, 1).expand(6, 1, 2, 8).contiguous()
    pages = nt.KVPages(k, k.clone())
    src, dst = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([4, 5], dtype=torch.int32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nt.nt_paged_copy(pages, src, dst)
    src.zero_(), dst.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert pages.k[:, 0, 0, 0].tolist() == [0, 1, 2, 3, 0, 1]


# ---- attention --------------------------------------------------------------

def _attn_case(nt, lens, page, H, Hk, d, dtype, seed=0, scale=None, edit=None, want_lse=True, wide=0):
    """``wide``: unused columns of the block table, which say how long the
    contexts may get (the call chooses its kernel by that)."""
    kp, vp, table = make_pool(lens, page, Hk, d, dtype, seed)
    table = torch.nn.functional.pad(table, (0, wide), value=-1)
    q = (2 * _rand(seed + 100, len(lens), H, d)).to(dtype)
    if edit:
        edit(kp, vp, table, q)
    pages = nt.KVPages(kp.to(DEV), vp.to(DEV))
    o, lse = nt.nt_paged_attn(pages, q.to(DEV), table.to(DEV), _i32(lens), scale=scale, want_lse=want_lse)
    nt.nt_device_status()
    return (kp, vp, table, q), o, lse


def _check(inputs, o, lse, lens, dtype, scale=None):
    kp, vp, table, q = inputs
    ro, rl, mag, cond = paged_attn(kp, vp, q, table, lens, scale)
    n = max(list(lens) + [0])
    err = (o.double().cpu() - ro).abs()
    bound = attn_bound(ro, mag, cond, n, dtype) + 1e-38
    assert bool((err <= bound).all()), float((err / bound).max())
    if lse is not None:
        empty = torch.tensor([x == 0 for x in lens])
        assert bool((lse.cpu()[:, empty] == -math.inf).all())
        # a score's error as in attn_bound, and the sum's: 64 + n / 8 steps
        lerr = (lse.double().cpu() - rl)[:, ~empty].abs()
        lb = (16 * cond[..., 0].T + 64 + n / 8 + 4 * rl.abs())[:, ~empty] * 2.0 ** -24
        assert bool((lerr <= lb).all()), float((lerr / lb).max())


SHAPES = [  # lens, page, H, Hk, d
    ([1], 16, 1, 1, 64),
    ([777], 16, 12, 12, 64),
    ([0], 16, 2, 1, 64),
    ([0, 5, 0, 64, 65, 0, 1, 130, 16, 0], 16, 8, 2, 64),
    ([63, 64, 65, 127, 128, 129, 15, 16, 17], 16, 8, 1, 128),
    ([300, 7, 0, 1000], 8, 4, 4, 128),
    ([300, 7, 0, 1000], 24, 14, 2, 128),          # 7 heads to a key head, pages of 24
    ([300, 41], 1, 2, 2, 32),
    ([513, 2], 7, 6, 2, 64),
    ([100, 700], 48, 32, 2, 64),                  # 16 heads to a key head
    ([100, 700], 256, 24, 1, 128),                # 24: more than one item per key head
    ([50, 3], 128, 40, 1, 64),
    ([2500], 64, 8, 1, 128),                      # one long sequence over many CTAs
    ([1] * 700, 16, 2, 1, 64),                    # more sequences than threads of a CTA
    ([3000, 1, 1, 2000, 5], 100, 5, 5, 32),
]


@pytest.mark.parametrize("room", ["exact", "1024", "wide"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_attn(nt, shape, dtype, room):
    """Every shape with a table as wide as its longest context, and with
    wider ones."""
    lens, page, H, Hk, d = shape
    wide = {"exact": 0, "1024": max(0, 1024 // page - -(-max(lens) // page)), "wide": -(-5000 // page)}[room]
    inputs, o, lse = _attn_case(nt, lens, page, H, Hk, d, dtype, wide=wide)
    _check(inputs, o, lse, lens, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] % 8 == 0])
def test_attn_long_tables(nt, shape, dtype):
    """Tables made for contexts of 200,000 positions: the kernel that long
    contexts take, at every shape."""
    lens, page, H, Hk, d = shape
    inputs, o, lse = _attn_case(nt, lens, page, H, Hk, d, dtype, wide=200000 // page)
    _check(inputs, o, lse, lens, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 10])
@pytest.mark.parametrize("B", [1, 2, 3, 5, 9, 20, 40, 90])
def test_attn_cluster_sizes(nt, B, page, dtype):
    """Batches of few items, which are spread over more CTAs the fewer they
    are; lengths around the slices' and the CTAs' ends."""
    lens = [[1, 15, 16, 17, 255, 256, 257, 0, 1000, 1553, 1537, 96, 97, 500][i % 14] for i in range(B - 1)] + [1600]
    inputs, o, lse = _attn_case(nt, lens, page, 8, 2, 64, dtype, seed=B)
    _check(inputs, o, lse, lens, dtype)


# contexts of a few positions, where a table of few pages is all there is
SHORT = [  # lens, page, H, Hk, d
    ([1, 0, 3, 16, 17, 128, 127, 64], 16, 12, 12, 64),
    ([5, 33, 0, 0, 90], 8, 32, 2, 128),              # 16 heads to a key head
    ([5, 33, 0, 0, 90], 24, 48, 2, 32),              # 24
    ([128] * 3, 128, 7, 1, 64),
    ([9, 100], 1, 3, 1, 64),                         # pages of one position
    ([9, 100, 31], 5, 10, 5, 32),
    ([1, 2, 3, 4] * 300, 2, 4, 2, 64),               # more items than warps
    ([0] * 5, 16, 8, 1, 128),
    ([77, 1, 120, 16, 15], 40, 6, 3, 128),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHORT)
def test_attn_short(nt, shape, dtype):
    lens, page, H, Hk, d = shape
    inputs, o, lse = _attn_case(nt, lens, page, H, Hk, d, dtype)
    _check(inputs, o, lse, lens, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page,lens,wide", [(16, [1, 5, 17, 70, 131], 400), (12, [1, 5, 17, 70, 131], 400),
                                            (16, [1, 5, 17, 70, 111], 0), (12, [1, 5, 17, 70, 111], 0)])
def test_attn_nothing_behind_the_end(nt, dtype, page, lens, wide):
    """NaN and infinities in the cache's rows behind the last position, in
    spare pages and in the table's unused entries reach no output."""

    def edit(kp, vp, table, q):
        used = torch.zeros(kp.shape[0], kp.shape[2], dtype=torch.bool)
        for b, n in enumerate(lens):
            for x in range(n):
                used[table[b, x // page], x % page] = True
        mask = ~used[:, None, :, None].expand_as(kp)
        kp[mask] = math.nan
        vp[mask] = math.inf
        vp[mask & (torch.arange(kp.shape[3]) % 2 == 0)] = math.nan
        table[table < 0] = 1 << 30

    inputs, o, lse = _attn_case(nt, lens, page, 8, 2, 64, dtype, edit=edit, wide=wide)
    _check(inputs, o, lse, lens, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_peaked_scores(nt, dtype):
    """Scores hundreds apart in rising and falling order: the running maximum
    moves at almost every key, or never after the first."""
    lens = [400, 400]

    def edit(kp, vp, table, q):
        q.fill_(1.0)
        for b in range(2):
            for x in range(lens[b]):
                s = (x if b == 0 else lens[b] - x) / 8.0
                kp[table[b, x // 16], :, x % 16] = s
    inputs, o, lse = _attn_case(nt, lens, 16, 4, 2, 64, dtype, edit=edit)
    _check(inputs, o, lse, lens, dtype)


def test_attn_strided_query_shared_pages_and_scale(nt):
    """q as a slice of a fused projection, two sequences on the same pages."""
    lens = [90, 90, 33]
    kp, vp, table = make_pool([90, 0, 33], 16, 2, 128, BF, 5)
    table[1] = table[0]
    x = _rand(7, 3, 12, 128, dtype=BF)
    pages = nt.KVPages(kp.to(DEV), vp.to(DEV))
    o, lse = nt.nt_paged_attn(pages, x.to(DEV)[:, 2:10], table.to(DEV), _i32(lens), scale=0.02, want_lse=True)
    _check((kp, vp, table, x[:, 2:10]), o, lse, lens, BF, scale=0.02)


def test_attn_empty_batch(nt):
    kp = torch.zeros(1, 2, 16, 64, device=DEV)
    o, _ = nt.nt_paged_attn(nt.KVPages(kp, kp), torch.zeros(0, 4, 64, device=DEV),
                            torch.zeros(0, 3, dtype=torch.int32, device=DEV), _i32([]))
    assert o.shape == (0, 4, 64)
    # a batch whose tables have no pages: every length must be 0
    o, _ = nt.nt_paged_attn(nt.KVPages(kp, kp), torch.ones(2, 4, 64, device=DEV),
                            torch.zeros(2, 0, dtype=torch.int32, device=DEV), _i32([0, 0]))
    nt.nt_device_status()
    assert int(torch.count_nonzero(o)) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length"])
@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("scale_up", [1, 30])
def test_attn_flags_bad_tables(nt, what, dtype, page, scale_up):
    """A page outside the pool reads as zeros, a length beyond the table as
    the table's, a negative one as 0; each is flagged and the other sequences
    keep their results."""
    lens = [40 * scale_up, 20 * scale_up]
    kp, vp, table = make_pool(lens, page, 1, 64, dtype, 3)
    q = _rand(4, 2, 2, 64, dtype=dtype)
    t2, l2 = table.clone(), list(lens)
    if what == "page":
        t2[0, 1] = kp.shape[0]
    elif what == "negative page":
        t2[0, 1] = -5
    elif what == "length":
        l2[0] = table.shape[1] * page + 1
    else:
        l2[0] = -1
    pages = nt.KVPages(kp.to(DEV), vp.to(DEV))
    o, _ = nt.nt_paged_attn(pages, q.to(DEV), t2.to(DEV), _i32(l2))
    with pytest.raises(nt.NTError) as ei:
        nt.nt_device_status()
    assert ei.value.status == 6
    ro, _, mag, cond = paged_attn(kp, vp, q, table, lens)
    err = (o.double().cpu() - ro).abs()[1]
    assert bool((err <= attn_bound(ro, mag, cond, max(lens), dtype)[1] + 1e-38).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cap", [900, 112])
def test_attn_captured_follows_lengths(nt, dtype, cap):
    """A captured call replayed with other lengths and queries gives what a
    direct call gives, bit for bit; a second captured call with a workspace
    of its own does too."""
    page, H, Hk, d = 16, 8, 2, 64
    kp, vp, table = make_pool([cap] * 3, page, Hk, d, dtype, 1)
    pages = nt.KVPages(kp.to(DEV), vp.to(DEV))
    table = table.to(DEV)
    q = torch.zeros(3, H, d, dtype=dtype, device=DEV)
    lens = _i32([1, 1, 1])
    ws = [torch.empty(nt.nt_paged_attn_workspace_bytes(H, Hk, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    nt.nt_paged_attn(pages, q, table, lens, workspace=ws[0])
    graphs, outs = [], []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(nt.nt_paged_attn(pages, q, table, lens, workspace=w, want_lse=True))
        graphs.append(g)
    for ls in ([900, 3, 0], [17, 900, 64], [0, 0, 0], [256, 255, 899]):
        lens.copy_(torch.tensor(ls, dtype=torch.int32).clamp(max=cap))
        q.normal_()
        for w in ws:
            w.fill_(255)
        for g in graphs:
            g.replay()
        want, wl = nt.nt_paged_attn(pages, q, table, lens, want_lse=True)
        for o, lse in outs:
            assert torch.equal(o, want) and torch.equal(lse, wl)


def test_attn_two_streams(nt):
    """Two calls at once on two streams, each with its own workspace."""
    lens = [700, 30, 0, 401]
    kp, vp, table = make_pool(lens, 16, 4, 128, BF, 8)
    pages = nt.KVPages(kp.to(DEV), vp.to(DEV))
    q = _rand(9, 4, 16, 128, dtype=BF).to(DEV)
    table, ln = table.to(DEV), _i32(lens)
    want, _ = nt.nt_paged_attn(pages, q, table, ln)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(want) for _ in streams]
    ws = [torch.empty(nt.nt_paged_attn_workspace_bytes(16, 4, 128), dtype=torch.uint8, device=DEV) for _ in streams]
    for _ in range(20):
        for s, o, w in zip(streams, outs, ws):
            nt.nt_paged_attn(pages, q, table, ln, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("d,page,H", [(128, 64, 8), (128, 16, 24), (64, 64, 8), (64, 8, 32)])
def test_attn_long_contexts_many_times(nt, d, page, H):
    """Contexts of tens of thousands of keys, bf16, repeated back to back on
    one workspace: every repeat gives the first one's bits, and those are
    right (fp64 on the device)."""
    lens, Hk = [70001, 40000, 3, 65536], 2
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = torch.zeros(4, max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    gen = torch.Generator(device=DEV).manual_seed(2)
    kp = torch.randn(at, Hk, page, d, generator=gen, device=DEV, dtype=BF)
    vp = torch.randn(at, Hk, page, d, generator=gen, device=DEV, dtype=BF)
    q = 2 * torch.randn(4, H, d, generator=gen, device=DEV, dtype=BF)
    pages, tab, ln = nt.KVPages(kp, vp), table.to(DEV), _i32(lens)
    ws = torch.empty(nt.nt_paged_attn_workspace_bytes(H, Hk, d), dtype=torch.uint8, device=DEV)
    outs = [nt.nt_paged_attn(pages, q, tab, ln, workspace=ws)[0] for _ in range(60)]
    nt.nt_device_status()
    assert all(torch.equal(o, outs[0]) for o in outs)
    for b, n in enumerate(lens):
        rows = tab[b, :need[b]].long()
        k = kp[rows].transpose(0, 1).reshape(Hk, -1, d)[:, :n].double()
        v = vp[rows].transpose(0, 1).reshape(Hk, -1, d)[:, :n].double()
        qb = q[b].double().reshape(Hk, -1, d)
        p = torch.softmax(qb @ k.transpose(1, 2) * d ** -0.5, -1)
        ro, mag = (p @ v).reshape(H, d).cpu(), (p @ v.abs()).reshape(H, d).cpu()
        cond = ((qb.abs() @ k.abs().transpose(1, 2)).amax(-1) * d ** -0.5).reshape(H, 1).cpu()
        err = (outs[0][b].double().cpu() - ro).abs()
        assert bool((err <= attn_bound(ro, mag, cond, n, BF)).all())


def test_attn_far_page_offsets(nt):
    """Pages behind 2^31 elements of the pool are addressed in full."""
    page, Hk, d = 256, 64, 128
    n_pages = (1 << 31) // (page * Hk * d) + 3                 # 2^31 elements and a little: 4.3 GB each
    k = torch.zeros(n_pages, Hk, page, d, dtype=BF, device=DEV)
    v = torch.zeros(n_pages, Hk, page, d, dtype=BF, device=DEV)
    far = n_pages - 1
    assert far * page * Hk * d > 2 ** 31
    new = _rand(1, 5, Hk, d, dtype=BF).to(DEV)
    pages = nt.KVPages(k, v)
    nt.nt_paged_write(pages, new, 2 * new, _i32([0, 5]), _i32([[far]]))
    q = _rand(2, 1, Hk, d, dtype=BF).to(DEV)
    o, _ = nt.nt_paged_attn(pages, q, _i32([[far]]), _i32([5]))
    nt.nt_paged_copy(pages, torch.tensor([far], dtype=torch.int32), torch.tensor([0], dtype=torch.int32))
    nt.nt_device_status()
    assert torch.equal(k[0], k[far]) and torch.equal(v[0], v[far])
    ro, _, mag, cond = paged_attn(k[far:].cpu(), v[far:].cpu(), q.cpu(), torch.tensor([[0]]), [5])
    assert bool(((o.double().cpu() - ro).abs() <= attn_bound(ro, mag, cond, 5, BF)).all())


@pytest.mark.parametrize("page,dtype", [(65536, BF), (65528, F32)])
def test_attn_longest_context(nt, page, dtype):
    """2^31 - 1 positions (one page many times over): counts of keys and tiles
    next to the end of 32 bits.  Against fp64 over the page's rows, each as
    often as it is attended to.  A sum of n roundings in turn is off by n
    steps of 2^-24 at most (2^-23 on the tensor cores, which may cut): a warp
    adds 32 lanes' keys in turn, 2^31 / (8 warps x 152) of them at most one by
    one (fp32), 16 at a time (bf16)."""
    n, d = 2 ** 31 - 1, 32
    k, v, q = (_rand(i, *s, dtype=dtype) for i, s in enumerate([(1, 1, page, d), (1, 1, page, d), (1, 1, d)]))
    v = v.abs()
    entries = -(-n // page)
    table = torch.zeros(1, entries, dtype=torch.int32, device=DEV)
    o, lse = nt.nt_paged_attn(nt.KVPages(k.to(DEV), v.to(DEV)), q.to(DEV), table, _i32([n]), want_lse=True)
    nt.nt_device_status()
    last = n - (entries - 1) * page                    # rows of the last page that count
    times = torch.full((page,), float(entries - 1), dtype=torch.float64)
    times[:last] += 1
    s = k[0, 0].double() @ q[0, 0].double() * d ** -0.5
    w = times * torch.exp(s - s.max())
    ro, rl = (w @ v[0, 0].double()) / w.sum(), float(s.max() + torch.log(w.sum()))
    added = n / (8 * 152) / (16 if dtype == BF else 1)
    rel = added * (2.0 ** -23 + 2.0 ** -24) + 2 * HALF_STEP[dtype]       # output and sum; P's and o's rounding in bf16
    assert bool(((o[0, 0].double().cpu() - ro).abs() <= rel * ro).all())
    assert abs(float(lse) - rl) <= rel
