"""nt_paged_tree_attn where it can go wrong, every kernel of it: values that are
not finite, rows that see nothing, refused lengths and pages, strides, streams,
captures, pools beyond 2^31 elements."""
import math

import numpy as np
import pytest
import torch

from _drafts import tree_attn
from test_gpu_drafts import BF, DEV, F32, _cu, _i32, call, call_kernel, check, make_case, nt  # noqa: F401

pytestmark = pytest.mark.gpu

KERNELS = ["call", 0, 1, 2, 3]
MIXED = dict(ctx=[0, 5, 100, 63, 0, 64, 300], ns=[3, 0, 7, 1, 40, 65, 9], page=16, H=8, Hk=2, d=64)
WIDE = dict(ctx=[0, 127, 128, 500], ns=[5, 64, 1, 130], page=24, H=6, Hk=2, d=128)
NARROW = dict(ctx=[0, 31, 200], ns=[9, 20, 3], page=8, H=4, Hk=1, d=32)


def by(nt, c, kernel, **kw):
    return call(nt, c, **kw) if kernel == "call" else call_kernel(nt, c, kernel, **kw)


def at(c, table, b, x):
    """Page and row of position x of sequence b."""
    ps = c["page"]
    return int(table[b, x // ps]), x % ps


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [MIXED, WIDE, NARROW])
@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_that_see_nothing(nt, kernel, shape, dtype):
    """Random masks, every third token's empty, and all of one sequence's:
    without a context those rows are 0, with one they are its attention."""
    def edit(kp, vp, table, q, bits):
        rng = np.random.default_rng(5)
        bits.copy_(torch.from_numpy(rng.integers(-2 ** 63, 2 ** 63 - 1, tuple(bits.shape))))
        bits[::3] = 0
        bits[:shape["ns"][0]] = 0

    c = make_case(**shape, dtype=dtype, seed=3, edit=edit)
    got = by(nt, c, kernel)
    if got:
        check(c, *got)
        assert bool((got[0][:shape["ns"][0]] == 0).all()) and bool((got[1][:, :shape["ns"][0]] == -math.inf).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [MIXED, WIDE, NARROW])
@pytest.mark.parametrize("kernel", KERNELS)
def test_masked_places_hold_anything(nt, kernel, shape, dtype):
    """Keys and values of drafted tokens that few rows see, and everything
    behind a sequence's end, are NaN or infinite: they reach the rows that see
    them, and no other."""
    def edit(kp, vp, table, q, bits):
        first = 0
        for b, (ctx, n) in enumerate(zip(shape["ctx"], shape["ns"])):
            L = ctx + n
            for x in range(L, table.shape[1] * shape["page"]):
                if int(table[b, x // shape["page"]]) < 0:
                    break
                page, row = at(shape, table, b, x)
                kp[page, :, row] = math.nan
                vp[page, :, row] = math.inf
            if n > 2:
                page, row = at(shape, table, b, L - 1)         # a token that nobody sees, not even itself
                kp[page, :, row], vp[page, :, row] = math.nan, math.nan
                w, s = divmod(n - 1, 64)
                bits[first:first + n, w] &= ~torch.tensor(1 << s if s < 63 else -2 ** 63)
                page, row = at(shape, table, b, L - 2)         # one that some see
                vp[page, 0, row, 3], vp[page, -1, row, 7] = math.inf, math.nan
            first += n

    c = make_case(**shape, dtype=dtype, seed=4, edit=edit)
    got = by(nt, c, kernel)
    if got:
        check(c, *got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel", KERNELS)
def test_context_values_not_finite(nt, kernel, dtype):
    """Every row of the sequence sees an infinite value in its context."""
    def edit(kp, vp, table, q, bits):
        page, row = at(MIXED, table, 2, 17)
        vp[page, 1, row, 5] = -math.inf

    c = make_case(**MIXED, dtype=dtype, seed=6, edit=edit)
    got = by(nt, c, kernel)
    if got:
        check(c, *got)
        assert bool((got[0][3:10, 4:, 5] == -math.inf).all()) and int(torch.isinf(got[0]).sum()) == 7 * 4


@pytest.mark.parametrize("kernel", KERNELS)
def test_scores_far_apart(nt, kernel):
    """Scores of +-10^4, so that maxima jump from tile to tile, and equal ones."""
    def edit(kp, vp, table, q, bits):
        kp *= torch.linspace(0, 60, kp.shape[0])[:, None, None, None].to(kp.dtype)
        q[::5] = 0

    c = make_case([700, 0, 260], [9, 33, 70], 16, 8, 2, 64, BF, seed=8, edit=edit)
    got = by(nt, c, kernel)
    if got:
        check(c, *got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cluster", range(1, 13))
def test_cluster_sizes(nt, cluster, dtype):
    c = make_case([0, 5, 333, 1000], [3, 7, 20, 1], 12, 4, 2, 64, dtype, seed=cluster)
    check(c, *call_kernel(nt, c, 3, cluster=cluster))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel", KERNELS)
def test_flags(nt, kernel, dtype):
    """Lengths, offsets and pages that do not fit are flagged; outputs of
    such sequences stay as they were, a bad page reads as zeros."""
    c = make_case([20, 30, 40, 50], [4, 4, 4, 4], 16, 4, 2, 64, dtype, seed=2)
    dev = {k: c[k].to(DEV) for k in ("q", "table", "bits")}
    pages = nt.KVPages(c["kp"].to(DEV), c["vp"].to(DEV))

    def run(cu, lens, table):
        out, lse = torch.full_like(dev["q"], 7), torch.full((4, 16), 7.0, device=DEV)
        args = (pages, dev["q"], _i32(cu), table, _i32(lens), 4)
        if kernel == "call":
            nt.nt_paged_tree_attn(*args, bits=dev["bits"], out=out, lse=lse)
        else:
            try:
                nt.nt_selftest_paged_tree_attn(kernel, *args, bits=dev["bits"], out=out, lse=lse)
            except nt.NTError as e:
                assert e.status == 2
                return None
        return out, lse

    good = run([0, 4, 8, 12, 16], c["lens"], dev["table"])
    nt.nt_device_status()
    if good is None:
        return
    width = 16 * dev["table"].shape[1]
    for cu, lens, bad in [([0, 4, 8, 12, 16], [24, 3, 44, 54], [1]), ([0, 4, 8, 12, 16], [24, -5, 44, width + 1], [1, 3]),
                          ([0, 4, 3, 12, 16], c["lens"], [1, 2]), ([0, 4, 8, 12, 17], c["lens"], [3]),
                          ([-1, 4, 8, 12, 16], c["lens"], [0]), ([0, 4, 9, 12, 16], [24, 34, 43, 54], [1])]:
        out, lse = run(cu, lens, dev["table"])
        with pytest.raises(nt.NTError) as e:
            nt.nt_device_status()
        assert e.value.status == 6
        for b in range(4):
            rows = slice(4 * b, 4 * b + 4)
            if b in bad:
                written = torch.zeros(16, dtype=torch.bool)
                for i in range(4):
                    if i not in bad and 0 <= cu[i] <= cu[i + 1] <= 16:
                        written[cu[i]:cu[i + 1]] = True
                keep = ~written[rows]
                assert bool((out[rows][keep] == 7).all()) and bool((lse[:, rows][:, keep] == 7).all())
            elif cu[b] == 4 * b and cu[b + 1] == 4 * b + 4 and lens[b] == c["lens"][b]:
                torch.testing.assert_close(out[rows].float(), good[0][rows].float(), rtol=2e-2, atol=2e-2)
    for page in (-1, c["kp"].shape[0], 2 ** 31 - 1, -2 ** 31):
        table = dev["table"].clone()
        table[1, 1] = page
        out, lse = run([0, 4, 8, 12, 16], c["lens"], table)
        with pytest.raises(nt.NTError):
            nt.nt_device_status()
        zero = dict(c, kp=c["kp"].clone(), vp=c["vp"].clone())
        zero["kp"][int(c["table"][1, 1])] = 0
        zero["vp"][int(c["table"][1, 1])] = 0
        check(zero, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel", KERNELS)
def test_strides_and_padding(nt, kernel, dtype):
    """Queries cut out of wider rows; tokens behind the last segment are left
    as they are, and may hold anything; max_new beyond what is there."""
    c = make_case([40, 0, 300], [5, 2, 30], 16, 4, 2, 64, dtype, seed=9, max_new=77)
    T, pad = 37, 11
    wide = torch.full((T + pad, 3 * 4 * 64 + 8), math.nan, dtype=dtype, device=DEV)
    q = wide[:, 8:8 + 256].unflatten(1, (4, 64))
    q[:T] = c["q"].to(DEV)
    bits = torch.full((T + pad, 2), -1, dtype=torch.int64, device=DEV)
    bits[:T] = c["bits"].to(DEV)
    out, lse = torch.full((T + pad, 4, 64), 7, dtype=dtype, device=DEV), torch.full((4, T + pad), 7.0, device=DEV)
    args = (nt.KVPages(c["kp"].to(DEV), c["vp"].to(DEV)), q, _cu(c["ns"]), c["table"].to(DEV), _i32(c["lens"]), 77)
    try:
        if kernel == "call":
            nt.nt_paged_tree_attn(*args, bits=bits, out=out, lse=lse)
        else:
            nt.nt_selftest_paged_tree_attn(kernel, *args, bits=bits, out=out, lse=lse)
    except nt.NTError as e:
        assert kernel != "call" and e.status == 2
        return
    nt.nt_device_status()
    check(c, out[:T], lse[:, :T])
    assert bool((out[T:] == 7).all()) and bool((lse[:, T:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel", [0, 1, 2, 3])
@pytest.mark.parametrize("B,ctx,n", [(200, 30, 3), (129, 100, 1), (1100, 2, 2)])
def test_many_sequences(nt, B, ctx, n, kernel, dtype):
    """More sequences than a warp plans, and than a CTA has threads."""
    rng = np.random.default_rng(B)
    c = make_case([int(x) for x in rng.integers(0, ctx + 1, B)], [int(x) for x in rng.integers(0, n + 1, B)], 8, 2, 1, 64,
                  dtype, seed=B)
    got = call_kernel(nt, c, kernel)
    if got:
        check(c, *got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel", [0, 1, 2, 3])
def test_few_items_with_many_parts(nt, kernel, dtype):
    """Single sequences split over all CTAs, whose results are joined."""
    for ctx, n, H, Hk in [(9000, 3, 1, 1), (9000, 53, 1, 1), (5000, 9, 2, 2), (20000, 1, 4, 1)]:
        c = make_case([ctx], [n], 32, H, Hk, 64, dtype, seed=n)
        got = call_kernel(nt, c, kernel)
        if got:
            check(c, *got)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_bits_every_time(nt, dtype):
    c = make_case([3000, 1, 1500], [40, 7, 1], 16, 8, 2, 64, dtype, seed=1)
    for kernel in KERNELS:
        first = by(nt, c, kernel)
        for _ in range(3):
            if first:
                again = by(nt, c, kernel)
                assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel", KERNELS)
def test_captured_follows_lengths(nt, kernel, dtype):
    """A captured call, replayed with other lengths, offsets, tables and
    masks, gives what a call with them gives."""
    c = [make_case(ctx, ns, 16, 8, 2, 64, dtype, seed=s, max_new=64)
         for s, (ctx, ns) in enumerate([([300, 20, 0], [8, 64, 8]), ([0, 900, 77], [30, 0, 50]), ([500, 0, 3], [0, 0, 1])])]
    width, n_pages = max(x["table"].shape[1] for x in c), max(x["kp"].shape[0] for x in c)
    pool = [torch.zeros(n_pages, 2, 16, 64, dtype=dtype, device=DEV) for _ in range(2)]
    pages = nt.KVPages(*pool)
    q, bits = torch.zeros(80, 8, 64, dtype=dtype, device=DEV), torch.zeros(80, 1, dtype=torch.int64, device=DEV)
    table, cu, lens = torch.zeros(3, width, dtype=torch.int32, device=DEV), _i32([0] * 4), _i32([0] * 3)
    ws = torch.empty(nt.nt_paged_tree_attn_workspace_bytes(8, 2, 64, 64), dtype=torch.uint8, device=DEV)

    def fill(x):
        n = x["q"].shape[0]
        pool[0][:x["kp"].shape[0]], pool[1][:x["vp"].shape[0]] = x["kp"].to(DEV), x["vp"].to(DEV)
        q[:n], bits[:n] = x["q"].to(DEV), x["bits"].to(DEV)
        table.fill_(-1)
        table[:, :x["table"].shape[1]] = x["table"].to(DEV)
        cu.copy_(_cu(x["ns"])), lens.copy_(_i32(x["lens"]))

    out, lse = torch.zeros_like(q), torch.zeros(8, 80, device=DEV)

    def run():
        kw = dict(bits=bits, out=out, lse=lse, workspace=ws)
        if kernel == "call":
            nt.nt_paged_tree_attn(pages, q, cu, table, lens, 64, **kw)
        else:
            nt.nt_selftest_paged_tree_attn(kernel, pages, q, cu, table, lens, 64, **kw)

    fill(c[0])
    try:
        run()
    except nt.NTError as e:
        assert kernel != "call" and e.status == 2
        return
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for x in c[1:] + c[:1]:
        fill(x)
        out.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        nt.nt_device_status()
        n = x["q"].shape[0]
        check(x, out[:n], lse[:, :n])
        again = out.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(out[:n], again[:n])


@pytest.mark.parametrize("kernel", [0, 1, 3])
def test_two_streams(nt, kernel):
    """Calls side by side with workspaces of their own."""
    cs = [make_case([4000 + 100 * s, 3], [30, 8], 16, 8, 2, 128, BF, seed=s) for s in range(2)]
    dev = [[x.to(DEV) for x in (c["kp"], c["vp"], c["q"], c["table"], c["bits"])] + [_cu(c["ns"]), _i32(c["lens"])]
           for c in cs]
    want = [call_kernel(nt, c, kernel)[0] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [torch.empty(nt.nt_paged_tree_attn_workspace_bytes(8, 2, 128, 30), dtype=torch.uint8, device=DEV) for _ in cs]
    outs = [[torch.empty_like(want[i]) for _ in range(20)] for i in range(2)]
    torch.cuda.synchronize()
    for k in range(20):
        for i, (kp, vp, q, table, bits, cu, lens) in enumerate(dev):
            nt.nt_selftest_paged_tree_attn(kernel, nt.KVPages(kp, vp), q, cu, table, lens, 30, bits=bits, out=outs[i][k],
                                           workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_far_pages(nt, kernel, dtype, d):
    """A pool of more than 2^31 elements, its last pages in use."""
    page, Hk = 16, 2
    n_pages = 2 ** 31 // (Hk * page * d) + 40
    c = make_case([200, 0], [7, 20], page, 4, Hk, d, dtype, seed=3)
    used = c["kp"].shape[0]
    kp = torch.empty(n_pages, Hk, page, d, dtype=dtype, device=DEV)
    vp = torch.empty(n_pages, Hk, page, d, dtype=dtype, device=DEV)
    kp[-used:], vp[-used:] = c["kp"].to(DEV), c["vp"].to(DEV)
    table = torch.where(c["table"] >= 0, c["table"] + n_pages - used, c["table"]).to(DEV)
    args = (nt.KVPages(kp, vp), c["q"].to(DEV), _cu(c["ns"]), table, _i32(c["lens"]), c["max_new"])
    try:
        if kernel == "call":
            o, lse = nt.nt_paged_tree_attn(*args, bits=c["bits"].to(DEV), want_lse=True)
        else:
            o, lse = nt.nt_selftest_paged_tree_attn(kernel, *args, bits=c["bits"].to(DEV))
    except nt.NTError as e:
        assert kernel != "call" and e.status == 2
        return
    nt.nt_device_status()
    check(c, o, lse)


def test_calls_on_another_stream(nt):
    """The calls of a drafted step queued on a side stream by argument, their
    results allocated by the call."""
    c = make_case([900, 3], [30, 8], 16, 8, 2, 64, BF, seed=2)
    want = call(nt, c)[0]
    kp, vp, q, table, bits = (c[k].to(DEV) for k in ("kp", "vp", "q", "table", "bits"))
    cu, lens = _cu(c["ns"]), _i32(c["lens"])
    parents = _i32([-1] * 38)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(10):
        got = nt.nt_paged_tree_attn(nt.KVPages(kp, vp), q, cu, table, lens, 30, bits=bits, stream=stream)[0]
        own, pos = nt.nt_draft_tree(parents, cu, 30, stream=stream)
        stream.synchronize()
        assert torch.equal(got, want) and pos.tolist() == [0] * 38
        assert own[:, 0].tolist() == [1 << i for i in range(30)] + [1 << i for i in range(8)]


def test_binding_refusals(nt):
    c = make_case([20, 3], [4, 2], 16, 4, 2, 64, BF, seed=2)
    kp, vp, q, table, bits = (c[k].to(DEV) for k in ("kp", "vp", "q", "table", "bits"))
    cu, lens, pages = _cu(c["ns"]), _i32(c["lens"]), nt.KVPages(kp, vp)
    good = dict(q=q, cu=cu, table=table, lengths=lens, max_new=4, bits=bits)

    def attend(**kw):
        a = {**good, **kw}
        extra = {k: a[k] for k in ("out", "lse", "workspace") if k in a}
        return nt.nt_paged_tree_attn(pages, a["q"], a["cu"], a["table"], a["lengths"], a["max_new"], bits=a["bits"], **extra)

    attend()
    refused = [dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q.cpu()), dict(cu=cu.long()), dict(cu=cu[:2]),
               dict(table=table.long()), dict(table=table[:1]), dict(table=table[0]), dict(lengths=lens[:1]),
               dict(lengths=lens.float()), dict(bits=bits.int()), dict(bits=bits[:, :0]), dict(bits=bits[:3]),
               dict(max_new=65), dict(max_new=-1), dict(max_new=257, bits=None), dict(out=torch.empty_like(q)[:3]),
               dict(out=torch.empty_like(q).float()), dict(lse=torch.empty(4, 5, device=DEV)),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV)), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))]
    for kw in refused:
        with pytest.raises((ValueError, nt.NTError)):
            attend(**kw)
    kept, pos0 = _i32([0]), _i32([20, 3])
    for call_ in (lambda: nt.nt_draft_tree(_i32([0] * 6).long(), cu, 4), lambda: nt.nt_draft_tree(_i32([-1] * 6), cu, 257),
                  lambda: nt.nt_draft_tree(_i32([-1] * 6), cu, 0), lambda: nt.nt_draft_tree(_i32([-1] * 6), cu, 4, pos0[:1]),
                  lambda: nt.nt_paged_keep(pages, kept.long(), _i32([0, 1, 1]), table, pos0),
                  lambda: nt.nt_paged_keep(pages, kept, _i32([0, 1]), table, pos0),
                  lambda: nt.nt_paged_keep(pages, kept, _i32([0, 1, 1]), table.cpu(), pos0),
                  lambda: nt.nt_paged_write_slots(pages, kp[0].transpose(0, 1), kp[0].transpose(0, 1), torch.zeros(3, dtype=torch.int64, device=DEV)),
                  lambda: nt.nt_paged_write_slots(pages, kp[:2, :, 0], vp[:2, :, 0], _i32([0, 1])),
                  lambda: nt.nt_paged_resize(table, lens, _i32([0]), _i32([0]), 0, lens, 0),
                  lambda: nt.nt_paged_resize(table, lens, _i32([0]), _i32([0]), 16, lens[:1], 0),
                  lambda: nt.nt_paged_resize(table, lens.long(), _i32([0]), _i32([0]), 16, lens, 0),
                  lambda: nt.nt_paged_resize(table, lens, _i32([0]), _i32([0]), 16, lens, -1)):
        with pytest.raises((ValueError, nt.NTError)):
            call_()
    nt.nt_device_status()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [MIXED, WIDE, NARROW])
@pytest.mark.parametrize("kernel", KERNELS)
def test_infinite_keys(nt, kernel, shape, dtype):
    """An infinite key in the context gives scores of -inf, weight 0, to the
    heads whose query is negative there, and NaN to the others."""
    b = max(i for i, (x, n) in enumerate(zip(shape["ctx"], shape["ns"])) if x > 4 and n)
    first, n = sum(shape["ns"][:b]), shape["ns"][b]

    def edit(kp, vp, table, q, bits):
        page, row = at(shape, table, b, 3)
        kp[page, 0, row, 2] = math.inf
        q[:, :, 2] = torch.where(q[:, :, 2] == 0, torch.ones_like(q[:, :, 2]), q[:, :, 2])

    c = make_case(**shape, dtype=dtype, seed=12, edit=edit)
    got = by(nt, c, kernel)
    if not got:
        return
    out = got[0].double().cpu()
    G = shape["H"] // shape["Hk"]
    up = torch.zeros(out.shape[:2], dtype=torch.bool)
    up[first:first + n, :G] = c["q"][first:first + n, :G, 2] > 0
    assert bool(torch.isnan(out[up]).all()) and bool(torch.isfinite(out[~up]).all())
    # the others as if the key were not there: a copy whose key gives them a score of -10^4 or less
    page, row = at(shape, c["table"], b, 3)
    far = dict(c, kp=c["kp"].clone())
    far["kp"][page, 0, row] = 0
    far["kp"][page, 0, row, 2] = 3e38
    plain = tree_attn(far["kp"], far["vp"], far["q"], far["ns"], far["table"], far["lens"], far["bits"])
    err, scale = (out - plain[0]).abs()[~up], plain[0].abs().max()
    assert float(err.max()) <= (2.0 ** -8 + 2.0 ** -12 if dtype == BF else 1e-5) * float(scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", range(8))
def test_sequences_of_one_and_two_row_tiles(nt, seed, d):
    """Tiles of sequences with more rows count for more when the batch is dealt
    out, so shares begin and end inside tiles: from fewer tiles than SMs to
    several to each."""
    rng = np.random.default_rng(seed)
    B = [1, 2, 5, 12, 30, 60, 150, 7][seed]
    ns = [int(x) for x in rng.choice([0, 1, 31, 32, 33, 64, 65, 200], B)]
    ctx = [int(x) for x in rng.integers(0, [3000, 900, 700, 500, 300, 200, 60, 5][seed], B)]
    ns[0] = 40
    c = make_case(ctx, ns, 16, 4, 1, d, BF, seed=seed)
    check(c, *call_kernel(nt, c, 1))
    check(c, *call(nt, c))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("kernel", KERNELS)
def test_pieces_of_prompts(nt, kernel, d, dtype):
    """No masks: items of a sequence's first tokens end before its last keys,
    wherever that is among tiles and shares."""
    for seed, (ctx, ns) in enumerate([([0], [256]), ([0, 1, 63, 127, 500], [256, 255, 129, 65, 64]),
                                      ([0] * 40, [200] * 40), ([2000, 3], [130, 256])]):
        c = make_case(ctx, ns, 16, 4, 1, d, dtype, kind="causal", seed=seed)
        got = by(nt, c, kernel)
        if got:
            check(c, *got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kernel", KERNELS)
def test_no_pages(nt, kernel, dtype):
    """A pool without pages: every page of the table is a bad one, read as zeros."""
    c = make_case([20, 0], [4, 2], 16, 4, 2, 64, dtype, seed=2)
    c["kp"], c["vp"] = c["kp"][:0], c["vp"][:0]
    pages = nt.KVPages(c["kp"].to(DEV), c["vp"].to(DEV))
    args = (pages, c["q"].to(DEV), _cu(c["ns"]), c["table"].to(DEV), _i32(c["lens"]), 4)
    try:
        if kernel == "call":
            out = nt.nt_paged_tree_attn(*args, bits=c["bits"].to(DEV))[0]
        else:
            out = nt.nt_selftest_paged_tree_attn(kernel, *args, bits=c["bits"].to(DEV))[0]
    except nt.NTError as e:
        assert kernel in (1, 2) and e.status == 2
        return
    with pytest.raises(nt.NTError) as e:
        nt.nt_device_status()
    assert e.value.status == 6 and bool((out == 0).all())
