"""Each of paged attention's kernels by name, at every size it takes: a warp
per item (0), a cluster of CTAs per item (1, of every size), tiles dealt out
to the SMs (2, with items kept whole where the tables are narrow, else cut and
joined).  The call chooses among them by the tables' width."""
import math

import pytest
import torch

from _attn_path import HALF_STEP, U32
from test_gpu_paged import BF, DEV, F32, SHAPES, SHORT, _i32, nt  # noqa: F401

pytestmark = pytest.mark.gpu

WARP, CLUSTER, TILES = 0, 1, 2


def _reference(kp, vp, q, table, lens, scale=None):
    """As _attn_path.paged_attn, in fp64 on the device, some sequences at a
    time, padded to the longest."""
    B, H, d = q.shape
    Hk, page = kp.shape[1], kp.shape[2]
    scale = d ** -0.5 if scale is None else scale
    o, mag = (torch.zeros(B, H, d, dtype=torch.float64, device=DEV) for _ in range(2))
    cond = torch.zeros(B, H, 1, dtype=torch.float64, device=DEV)
    lse = torch.full((H, B), -math.inf, dtype=torch.float64, device=DEV)
    some = [b for b in range(B) if lens[b] > 0]
    at_once = max(1, (1 << 26) // (Hk * d * max(list(lens) + [1])))
    for i in range(0, len(some), at_once):
        bs = some[i:i + at_once]
        n = torch.tensor([lens[b] for b in bs], device=DEV)
        x = torch.arange(int(n.max()), device=DEV)
        there = x < n[:, None]                                            # (b, x)
        ids = table[bs][:, x // page].long().where(there, 0)
        k, v = (t[ids, :, x % page].double() * there[..., None, None] for t in (kp, vp))
        qb = q[bs].double().reshape(len(bs), Hk, -1, d)
        s = torch.einsum("bjgd,bxjd->bjgx", qb, k) * scale
        s = s.masked_fill(~there[:, None, None], -math.inf)
        p = torch.softmax(s, -1)
        o[bs] = torch.einsum("bjgx,bxjd->bjgd", p, v).reshape(-1, H, d)
        mag[bs] = torch.einsum("bjgx,bxjd->bjgd", p, v.abs()).reshape(-1, H, d)
        cond[bs] = torch.einsum("bjgd,bxjd->bjgx", qb.abs(), k.abs()).amax(-1).reshape(-1, H, 1) * scale
        lse[:, bs] = torch.logsumexp(s, -1).reshape(-1, H).T
    return o, lse, mag, cond


def _check(ref, o, lse, lens, dtype):
    """The output's own rounding; of each probability 2^-15 in bf16; fp32
    steps: a score's 16 of its sum |q k| scale, twice (above and below the
    fraction bar), 16 for the exponential and the scale, six for every sixteen
    keys that a warp adds in turn (a factor, and two sums or products that the
    tensor cores may cut), 64 for the joins."""
    ro, rl, mag, cond = ref
    n = max(list(lens) + [0])
    turn = 6 * n / 16 + 64
    p = 2.0 ** -15 if dtype == BF else 0.0
    bound = HALF_STEP[dtype] * ro.abs() * 1.001 + (p + (32 * cond + 16 + turn) * U32) * mag + 1e-38
    err = (o.double() - ro).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    empty = torch.tensor([x == 0 for x in lens], device=DEV)
    assert bool((lse[:, empty] == -math.inf).all()) and int(torch.count_nonzero(o[empty])) == 0
    lerr = (lse.double() - rl)[:, ~empty].abs()
    lb = ((16 * cond[..., 0].T + 16 + turn + 4 * rl.abs()) * U32)[:, ~empty]
    assert bool((lerr <= lb).all()), float((lerr / lb).max())


def _inputs(lens, page, H, Hk, d, dtype, seed=0, wide=0):
    """Pages in random order, three of them spare, a table with -1 behind the
    ends and ``wide`` columns more, queries."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = torch.tensor([-(-n // page) for n in lens], device=DEV)
    pool = int(need.sum()) + 3
    used = torch.arange(max(1, int(need.max())) + wide, device=DEV) < need[:, None]
    table = torch.full(used.shape, -1, dtype=torch.int32, device=DEV)
    table[used] = torch.randperm(pool, generator=g, device=DEV)[:pool - 3].to(torch.int32)
    kp, vp = (torch.randn(pool, Hk, page, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    return kp, vp, table, (2 * torch.randn(len(lens), H, d, generator=g, device=DEV)).to(dtype)


def _run(nt, kernel, lens, page, H, Hk, d, dtype, seed=0, wide=0, cluster=0):  # noqa: F811
    kp, vp, table, q = _inputs(lens, page, H, Hk, d, dtype, seed, wide)
    o, lse = nt.nt_selftest_paged_attn(kernel, nt.KVPages(kp, vp), q, table, _i32(lens), cluster=cluster)
    nt.nt_device_status()
    _check(_reference(kp, vp, q, table, lens), o, lse, lens, dtype)


def _ragged(B, top, seed):
    """B lengths of 0 to top, some of them 0, 1, top and around the slices' ends."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, top + 1, (B,), generator=g).tolist()
    for i, n in enumerate((0, 1, 15, 16, 17, top, top, 0, 31, 33)):
        if i < B:
            lens[i * 7 % B] = min(n, top)
    return lens


# ---- a warp per item -----------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHORT + [s for s in SHAPES if max(s[0]) <= 1000])
def test_warps(nt, shape, dtype):  # noqa: F811
    lens, page, H, Hk, d = shape
    wide = min(3, 1024 // page - max(1, -(-max(lens) // page)))
    _run(nt, WARP, lens, page, H, Hk, d, dtype, wide=max(0, wide))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 7, 8, 12, 16, 24])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_warps_full(nt, d, G, dtype):  # noqa: F811
    """More items than the GPU has warps for, so that each takes several and
    copies the next one's keys under the present one's; pages of 1, 3 and 16,
    tables of more than 32 entries."""
    for i, page in enumerate((16, 3, 1)):
        Hk = (5, 2, 3)[i]
        lens = _ragged((700, 1600, 1100)[i], (200, 90, 60)[i], seed=G)
        _run(nt, WARP, lens, page, G * Hk, Hk, d, dtype, seed=i)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 1000])
def test_warps_long(nt, page, dtype):  # noqa: F811
    """Contexts up to the kernel's 1,024 positions."""
    top = 1024 // page * page
    _run(nt, WARP, _ragged(300, top, seed=page) + [top], page, 16, 8, 64, dtype)


# ---- clusters ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cluster", [0, 1, 5, 12])
@pytest.mark.parametrize("shape", SHAPES + SHORT)
def test_clusters(nt, shape, cluster, dtype):  # noqa: F811
    lens, page, H, Hk, d = shape
    _run(nt, CLUSTER, lens, page, H, Hk, d, dtype, cluster=cluster)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cluster", [1, 3, 12])
@pytest.mark.parametrize("d,G", [(32, 1), (64, 3), (64, 16), (128, 4), (128, 12)])
def test_clusters_of_many_items(nt, d, G, cluster, dtype):  # noqa: F811
    """More items than clusters run at once."""
    _run(nt, CLUSTER, _ragged(300, 700, seed=G), 12, G * 2, 2, d, dtype, cluster=cluster)


# ---- tiles ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("wide", [0, 400000])
@pytest.mark.parametrize("shape", [s for s in SHAPES + SHORT if s[1] % 8 == 0])
def test_tiles(nt, shape, wide, dtype):  # noqa: F811
    """Narrow tables, whose items are kept whole, and wide ones, whose items
    are cut."""
    lens, page, H, Hk, d = shape
    _run(nt, TILES, lens, page, H, Hk, d, dtype, wide=wide // page)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("wide", [0, 400000])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 7, 8, 12, 16, 24])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_tiles_full(nt, d, G, wide, dtype):  # noqa: F811
    """Hundreds of ragged contexts: many segments to a CTA, and items cut
    anywhere."""
    for i, (page, top) in enumerate(((16, 200), (8, 90), (24, 1500 if wide else 200))):
        Hk = (5, 2, 3)[i]
        _run(nt, TILES, _ragged((400, 700, 90)[i], top, seed=G), page, G * Hk, Hk, d, dtype, seed=i, wide=wide // page)


# ---- what each does with bad tables ---------------------------------------------------

KERNELS = [(WARP, 0), (CLUSTER, 0), (TILES, 0), (TILES, 400000)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("what", ["page", "negative page", "far page", "length", "longest length", "negative length"])
@pytest.mark.parametrize("kernel,wide", KERNELS)
def test_bad_tables(nt, kernel, wide, what, dtype):  # noqa: F811
    """A page outside the pool reads as zeros, a length beyond the table as
    the table's, a negative one as 0; each is flagged."""
    page, lens = 16, [200, 90, 400]
    kp, vp, table, q = _inputs(lens, page, 6, 2, 64, dtype, wide=wide // page)
    pool, right, n = kp.shape[0], table.clone(), list(lens)
    if "page" in what:
        table[0, 1] = {"page": pool, "negative page": -5, "far page": 2 ** 31 - 1}[what]
        kz, vz = (torch.cat((x, torch.zeros_like(x[:1]))) for x in (kp, vp))
        right[0, 1] = pool
    else:
        # behind its own pages the row goes on with others, so that the longest length can be read
        right[0, 13:] = table[0, 13:] = torch.arange(table.shape[1] - 13, dtype=torch.int32, device=DEV) % pool
        kz, vz = kp, vp
        n[0] = {"length": table.shape[1] * page + 1, "longest length": 2 ** 31 - 1, "negative length": -7}[what]
    o, lse = nt.nt_selftest_paged_attn(kernel, nt.KVPages(kp, vp), q, table, _i32(n))
    with pytest.raises(nt.NTError) as ei:
        nt.nt_device_status()
    assert ei.value.status == 6
    read = [min(max(x, 0), right.shape[1] * page) for x in n]
    _check(_reference(kz, vz, q, right, read), o, lse, read, dtype)


# ---- graphs, streams -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel,wide", KERNELS)
def test_captured_follows_lengths(nt, kernel, wide, dtype):  # noqa: F811
    """Two captured calls with a workspace each, replayed with other lengths
    (which cut other items), other queries and full workspaces, side by side:
    a direct call's bits."""
    cap, page, H, Hk, d = 1008, 16, 8, 2, 64
    kp, vp, table, q = _inputs([cap] * 3, page, H, Hk, d, dtype, wide=wide // page)
    pages, lens = nt.KVPages(kp, vp), _i32([1, 1, 1])
    ws = [torch.empty(nt.nt_paged_attn_workspace_bytes(H, Hk, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    call = lambda w=None: nt.nt_selftest_paged_attn(kernel, pages, q, table, lens, workspace=w)
    call(ws[0])
    graphs, outs = [], []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(w))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ws]
    for ls in ([1008, 3, 0], [17, 1000, 64], [0, 0, 0], [256, 255, 899], [1, 1, 1], [1008] * 3, [640, 1, 641]):
        lens.copy_(torch.tensor(ls, dtype=torch.int32))
        q.normal_()
        for w in ws:
            w.fill_(255)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        want = call()
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        _check(_reference(kp, vp, q, table, ls), *want, ls, dtype)
    nt.nt_device_status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel,wide", KERNELS)
def test_streams_at_once(nt, kernel, wide, dtype):  # noqa: F811
    """Calls on three streams at once, each with a workspace of its own, over
    and over: every one the first's bits."""
    lens, page, H, Hk, d = [1000, 30, 0, 401, 990, 16], 16, 16, 4, 128
    kp, vp, table, q = _inputs(lens, page, H, Hk, d, dtype, wide=wide // page)
    pages, n = nt.KVPages(kp, vp), _i32(lens)
    want = nt.nt_selftest_paged_attn(kernel, pages, q, table, n)
    _check(_reference(kp, vp, q, table, lens), *want, lens, dtype)
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws = [torch.full((nt.nt_paged_attn_workspace_bytes(H, Hk, d),), 255, dtype=torch.uint8, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for _ in range(25):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                outs.append(nt.nt_selftest_paged_attn(kernel, pages, q, table, n, workspace=w, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for got in outs for a, b in zip(got, want))
    nt.nt_device_status()


# ---- the longest context ----------------------------------------------------------------

@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("page,dtype", [(65536, BF), (65528, F32)])
def test_every_place_of_the_longest_context(nt, page, dtype, d):  # noqa: F811
    """2^31 - 1 positions, of which d attend to: the first, the last, those
    around 2^30 and on both sides of the CTAs' shares.  Each has the score 0
    and the value 1 in a column of its own, all others the score -64, whose
    sum is below 2^31 e^-64 = 3e-19: every output is 1 / d and the log-sum-exp
    log d, and a place that is missed, or taken twice, shows."""
    n, tile = 2 ** 31 - 1, {(BF, 32): 128, (BF, 128): 64, (F32, 32): 128, (F32, 128): 32}[dtype, d]
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    units = -(-n // tile) + 2                               # an item counts as two tiles more, in front
    places = [0, 2 ** 30 - 1, 2 ** 30, n - 1]
    step = ctas / (d / 2 - 2)                               # (d - 4) / 2 of the shares' ends
    for i in range((d - 4) // 2):
        at = (units * min(ctas - 1, max(1, round((i + 0.5) * step))) // ctas - 2) * tile
        places += [at - 1, at]
    assert len(set(places)) == d and max(places) < n
    entries = -(-n // page)
    special = sorted({x // page for x in places})
    table = torch.zeros(1, entries, dtype=torch.int32, device=DEV)
    k = torch.zeros(1 + len(special), 1, page, d, dtype=dtype, device=DEV)
    v = torch.zeros_like(k)
    k[..., 0] = -8.0
    for i, e in enumerate(special):
        table[0, e] = 1 + i
    for c, x in enumerate(places):
        i = 1 + special.index(x // page)
        k[i, 0, x % page, 0] = 0
        v[i, 0, x % page, c] = 1
    q = torch.zeros(1, 1, d, dtype=dtype, device=DEV)
    q[..., 0] = 8
    end = n - (entries - 1) * page                          # rows behind the last position
    k[-1, 0, end:], v[-1, 0, end:] = 8, math.nan
    o, lse = nt.nt_paged_attn(nt.KVPages(k, v), q, table, _i32([n]), scale=1.0, want_lse=True)
    nt.nt_device_status()
    # probabilities of exactly 1, sums of at most d of them: exact but for the others', the quotient and the logarithm
    assert float((o.double() - 1 / d).abs().max()) <= 4 * 2.0 ** -24 / d
    assert abs(float(lse) - math.log(d)) <= 8 * 2.0 ** -24 * math.log(d)
