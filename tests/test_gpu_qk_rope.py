"""nt_qk_norm_rope and its backward against the 64-bit plain form: both
layouts, part of the head, scaled frequencies, far positions, norms on either
side or none, shared key heads, strided and in-place tensors, one token to
thousands.

Bound: one rounding to the I/O type (half a step of the value) plus fp32
steps of the pair's magnitude: the mean of squares (at most 24 steps, halved
by the root), the root and reciprocal (4), the two products with r and gamma
(2), cosine and sine (angle 2, function 2, scale 1), two products and a sum
(3): below 32 steps of |y_a| + |y_b|."""
import math

import pytest
import torch

from _attn_path import HALF_STEP, U32, columns, inv_freq, positions_of, rope

pytestmark = pytest.mark.gpu

DEV = "cuda"
STEPS = 32


@pytest.fixture(scope="module")
def nt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_batching_gb300 import build, nt as ntmod
    build.build()
    return ntmod


def _rand(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def _cu(segs):
    return torch.tensor([0] + torch.tensor(segs).cumsum(0).tolist() if segs else [0], dtype=torch.int32, device=DEV)


def _close(got, ref, mag, dtype, steps=STEPS):
    err = (got.double().cpu() - ref).abs()
    bound = HALF_STEP[dtype] * ref.abs() * 1.001 + steps * U32 * mag + 1e-38
    assert bool((err <= bound).all()), float((err / bound).max())


CASES = [
    # segs, starts, H, Hk, d, rot, interleaved, norm q, norm k, scaling, rot_scale
    ([1], None, 1, 1, 16, 16, False, True, True, {}, 1.0),
    ([1] * 16, list(range(100000, 100016)), 32, 8, 128, 128, False, True, True,
     dict(scaling="bands", factor=4.0, original_len=32768, base=1e6), 1.1386),
    ([5, 0, 1, 130, 0, 64], None, 12, 12, 64, 64, False, True, True, {}, 1.0),
    ([5, 0, 1, 130, 0, 64], [0, 7, 3, 1000000, 5, 2**31 - 100], 4, 2, 64, 32, True, False, False,
     dict(scaling="linear", factor=8.0), 1.0),
    ([33, 700], None, 6, 2, 80, 48, False, True, False, dict(scaling="ntk", factor=2.0), 1.0),
    ([33, 200], None, 3, 1, 96, 96, True, False, True, {}, 1.0),
    ([40], None, 2, 2, 256, 64, True, True, True, {}, 0.7),
    ([77, 3], None, 7, 0, 32, 32, False, True, False, {}, 1.0),       # queries only
    ([77, 3], None, 0, 5, 32, 16, True, False, True, {}, 1.0),        # keys only
    ([3000, 1, 2048], None, 5, 1, 64, 64, False, True, True, {}, 1.0),
    ([1] + [0] * 70 + [2, 0, 1, 3] + [0] * 33 + [1] * 90 + [0] * 1200 + [5], None, 2, 1, 32, 32, False, True, True, {}, 1.0),
    ([1] * 1500, list(range(1500)), 1, 1, 16, 16, True, False, True, {}, 1.0),   # 32 tokens, 32 segments a warp
]


def _setup(case, dtype, seed=0):
    segs, starts, H, Hk, d, rot, inter, nq, nk, sc, rs = case
    T = sum(segs)
    q = _rand(seed, T, H, d, dtype=dtype) if H else None
    k = _rand(seed + 1, T, Hk, d, dtype=dtype) if Hk else None
    qg = 1 + 0.3 * _rand(seed + 2, d) if nq else None
    kg = 1 + 0.3 * _rand(seed + 3, d) if nk else None
    return q, k, qg, kg, positions_of(segs, starts), inv_freq(rot, **sc)


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_forward(nt, case, dtype):
    segs, starts, H, Hk, d, rot, inter, nq, nk, sc, rs = case
    q, k, qg, kg, pos, freq = _setup(case, dtype)
    turns = nt.nt_rope_turns(rot, device=DEV, **sc)
    p0 = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    qd, kd, qgd, kgd = _dev(q, k, qg, kg)
    qo, ko = nt.nt_qk_norm_rope(qd, kd, turns, cu_seqlens=_cu(segs), pos0=p0, q_gamma=qgd, k_gamma=kgd,
                                interleaved=inter, rot_scale=rs)
    nt.nt_device_status()
    for x, g, out in ((q, qg, qo), (k, kg, ko)):
        if x is None:
            assert out is None
            continue
        _close(out, *rope(x, pos, freq, g, 1e-6, inter, rs), dtype)
    # explicit positions: the same bits
    qo2, ko2 = nt.nt_qk_norm_rope(qd, kd, turns, positions=pos.to(torch.int32).to(DEV), q_gamma=qgd, k_gamma=kgd,
                                  interleaved=inter, rot_scale=rs)
    for a, b in ((qo, qo2), (ko, ko2)):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_only(nt, dtype):
    q = _rand(5, 19, 3, 48, dtype=dtype)
    g = 1 + _rand(6, 48)
    out, _ = nt.nt_qk_norm_rope(q.to(DEV), None, None, q_gamma=g.to(DEV), eps=1e-5)
    y, mag = rope(q, torch.zeros(19), None, g, 1e-5)
    _close(out, y, mag, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_fused_projection_slices_and_in_place(nt, dtype):
    """q and k as slices of one (T, (H + 2 Hk) d) projection, read in place,
    then rotated in place: v's columns and the neighbours stay as they were."""
    T, H, Hk, d = 37, 6, 2, 64
    segs = [30, 7]
    x = _rand(9, T, H + 2 * Hk, d, dtype=dtype).to(DEV)
    g = (1 + 0.1 * _rand(10, d)).to(DEV)
    turns = nt.nt_rope_turns(d, device=DEV)
    cu = _cu(segs)
    q, k = x[:, :H], x[:, H:H + Hk]
    qo, ko = nt.nt_qk_norm_rope(q, k, turns, cu_seqlens=cu, q_gamma=g, k_gamma=g)
    want = nt.nt_qk_norm_rope(q.contiguous(), k.contiguous(), turns, cu_seqlens=cu, q_gamma=g, k_gamma=g)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    v = x[:, H + Hk:].clone()
    nt.nt_qk_norm_rope(q, k, turns, cu_seqlens=cu, q_gamma=g, k_gamma=g, q_out=q, k_out=k)
    assert torch.equal(x[:, :H], qo) and torch.equal(x[:, H:H + Hk], ko) and torch.equal(x[:, H + Hk:], v)


def test_empty(nt):
    z = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    turns = nt.nt_rope_turns(64, device=DEV)
    qo, ko = nt.nt_qk_norm_rope(z, z, turns, cu_seqlens=_cu([]))
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 4, 64)
    g = torch.ones(64, device=DEV)
    out = nt.nt_qk_norm_rope_bwd(z, z, turns, q=z, k=z, cu_seqlens=_cu([0, 0]), q_gamma=g, k_gamma=g)
    assert float(out[2].abs().sum()) == 0 and float(out[3].abs().sum()) == 0


def test_bad_offsets_flagged_and_not_written(nt):
    """cu_seqlens that end before T: the tokens behind are flagged and their
    outputs untouched."""
    q = torch.ones(8, 1, 32, device=DEV)
    out = torch.full_like(q, 7.0)
    turns = nt.nt_rope_turns(32, device=DEV)
    nt.nt_qk_norm_rope(q, None, turns, cu_seqlens=torch.tensor([0, 5], dtype=torch.int32, device=DEV), q_out=out)
    with pytest.raises(nt.NTError) as ei:
        nt.nt_device_status()
    assert ei.value.status == 6
    assert bool((out[5:] == 7.0).all()) and bool((out[:5] != 7.0).all())


def test_nan_rows_stay_in_their_row(nt):
    q = _rand(1, 9, 2, 64)
    q[4, 1, 3] = math.nan
    q[7, 0, 0] = math.inf
    out, _ = nt.nt_qk_norm_rope(q.to(DEV), None, nt.nt_rope_turns(64, device=DEV), cu_seqlens=_cu([9]),
                                q_gamma=torch.ones(64, device=DEV))
    bad = torch.isnan(out.cpu()).any(-1)
    assert bad[4, 1] and bad[7, 0] and int(bad.sum()) == 2


@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_stay_in_their_pair(nt, interleaved):
    """Without a norm a column mixes with its pair's other column only, and
    one behind the rotated part with none, in both directions."""
    q = _rand(1, 5, 1, 64)
    q[0, 0, 40] = math.inf
    q[1, 0, 50] = -math.inf
    q[2, 0, 3] = math.nan
    a, b = columns(32, interleaved)
    pair = {int(x): int(y) for x, y in zip(a, b)} | {int(y): int(x) for x, y in zip(a, b)}
    turns = nt.nt_rope_turns(32, device=DEV)
    pos = torch.arange(1, 6, dtype=torch.int32, device=DEV)
    fwd = nt.nt_qk_norm_rope(q.to(DEV), None, turns, positions=pos, interleaved=interleaved)[0].cpu()
    bwd = nt.nt_qk_norm_rope_bwd(q.to(DEV), None, turns, positions=pos, interleaved=interleaved)[0].cpu()
    for out in (fwd, bwd):
        assert out[0, 0, 40] == math.inf and out[1, 0, 50] == -math.inf
        bad = ~torch.isfinite(out)
        assert bad[2].nonzero()[:, 1].tolist() == sorted((3, pair[3])) and int(bad.sum()) == 4


# Backward: g is off by 8 steps of its pair's |.| + |.| (as above without the
# norm), x r by 16 of itself, the mean of h x r by 16 + 8 + 24 steps of
# mean |h x r|; dx then by 64 steps of r (|h|_pair + |x r| mean |h x r|) at
# most.  dgamma: n rows of which each thread adds at most n / 64 + 24 in turn,
# after 24 steps a term: (n / 64 + 64) steps of sum |g x r|.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_backward(nt, case, dtype):
    segs, starts, H, Hk, d, rot, inter, nq, nk, sc, rs = case
    q, k, qg, kg, pos, freq = _setup(case, dtype, seed=20)
    T = sum(segs)
    dq = _rand(30, T, H, d, dtype=dtype) if H else None
    dk = _rand(31, T, Hk, d, dtype=dtype) if Hk else None
    turns = nt.nt_rope_turns(rot, device=DEV, **sc)
    p0 = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    dqd, dkd, qd, kd, qgd, kgd = _dev(dq, dk, q, k, qg, kg)
    run = lambda: nt.nt_qk_norm_rope_bwd(dqd, dkd, turns, q=qd, k=kd, cu_seqlens=_cu(segs), pos0=p0, q_gamma=qgd,
                                         k_gamma=kgd, interleaved=inter, rot_scale=rs)
    got = run()
    nt.nt_device_status()
    for x, u, g, out, dg in ((q, dq, qg, got[0], got[2]), (k, dk, kg, got[1], got[3])):
        if u is None:
            assert out is None
            continue
        # the transposed rotation is the rotation by minus the position
        gb, gmag = rope(u, -pos, freq, None, 0.0, inter, rs)
        if g is None:
            assert dg is None
            _close(out, gb, gmag, dtype)
            continue
        xf = x.double()
        r = 1 / torch.sqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
        n = xf * r
        h = gb * g.double()
        dx = r * (h - n * (h * n).mean(-1, keepdim=True))
        mag = r * (gmag * g.double().abs() + n.abs() * (gmag * g.double().abs() * n.abs()).mean(-1, keepdim=True))
        _close(out, dx, mag, dtype, steps=64)
        rows = x.shape[0] * x.shape[1]
        err = (dg.double().cpu() - (gb * n).sum((0, 1))).abs()
        bound = (rows / 64 + 64) * U32 * (gmag * n.abs()).sum((0, 1))
        assert bool((err <= bound).all()), float((err / bound).max())
    again = run()
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))      # bit-reproducible


def test_backward_against_differences(nt):
    """Directional derivative of sum(w out) by central differences in fp64 of
    the plain form, against the fp32 kernel's gradients."""
    segs, H, Hk, d = [3, 5], 2, 1, 32
    q, k = _rand(1, 8, H, d), _rand(2, 8, Hk, d)
    qg, kg = 1 + 0.2 * _rand(3, d), 1 + 0.2 * _rand(4, d)
    wq, wk = _rand(5, 8, H, d), _rand(6, 8, Hk, d)
    pos, freq = positions_of(segs), inv_freq(16)
    dq, dk, dqg, dkg = nt.nt_qk_norm_rope_bwd(*_dev(wq, wk), nt.nt_rope_turns(16, device=DEV), q=q.to(DEV),
                                              k=k.to(DEV), cu_seqlens=_cu(segs), q_gamma=qg.to(DEV),
                                              k_gamma=kg.to(DEV), interleaved=True)

    def f(q_, k_, qg_, kg_):
        return float((wq.double() * rope(q_, pos, freq, qg_, 1e-6, True)[0]).sum()
                     + (wk.double() * rope(k_, pos, freq, kg_, 1e-6, True)[0]).sum())

    args = [t.double() for t in (q, k, qg, kg)]
    for i, g in enumerate((dq, dk, dqg, dkg)):
        v = _rand(40 + i, *args[i].shape).double()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * v, args[i] - 1e-5 * v
        num = (f(*up) - f(*down)) / 2e-5
        ana = float((g.double().cpu() * v).sum())
        # differences of order h^2 = 1e-10 of third derivatives of order one,
        # summed over 8 H d terms; fp32 gradients: 64 steps of sum |g v|
        assert abs(num - ana) <= 1e-6 * (1 + float((g.double().cpu() * v).abs().sum()))


def test_backward_needs_no_inputs_without_norm(nt):
    u = _rand(3, 10, 2, 64, dtype=torch.bfloat16).to(DEV)
    turns = nt.nt_rope_turns(64, device=DEV)
    fwd = nt.nt_qk_norm_rope(u, None, turns, positions=torch.arange(10, dtype=torch.int32, device=DEV))[0]
    back = nt.nt_qk_norm_rope_bwd(u, None, turns, positions=-torch.arange(10, dtype=torch.int32, device=DEV))[0]
    # rotating back by minus the position is rotating forward
    assert torch.equal(fwd, back)


def test_captured_and_replayed(nt):
    """A captured forward and backward follow new inputs and starts."""
    T, H, Hk, d = 6, 4, 2, 64
    q = torch.empty(T, H, d, dtype=torch.bfloat16, device=DEV)
    k = torch.empty(T, Hk, d, dtype=torch.bfloat16, device=DEV)
    cu, p0 = _cu([1] * T), torch.zeros(T, dtype=torch.int32, device=DEV)
    g = torch.ones(d, device=DEV)
    turns = nt.nt_rope_turns(d, device=DEV)
    call = lambda: (nt.nt_qk_norm_rope(q, k, turns, cu_seqlens=cu, pos0=p0, q_gamma=g, k_gamma=g)
                    + nt.nt_qk_norm_rope_bwd(q, k, turns, q=q, k=k, cu_seqlens=cu, pos0=p0, q_gamma=g, k_gamma=g))
    q.normal_(), k.normal_()
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for i in range(3):
        q.normal_(), k.normal_()
        p0.fill_(1000 * i)
        graph.replay()
        got = [t.clone() for t in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_side_stream(nt):
    q = torch.randn(50, 4, 64, device=DEV)
    turns = nt.nt_rope_turns(64, device=DEV)
    cu = _cu([50])
    want = nt.nt_qk_norm_rope(q, None, turns, cu_seqlens=cu)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    nt.nt_qk_norm_rope(q, None, turns, cu_seqlens=cu, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_layout_columns():
    a, b = columns(8, True)
    assert a.tolist() == [0, 2, 4, 6] and b.tolist() == [1, 3, 5, 7]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", range(16, 257, 16))
def test_every_width(nt, d, dtype):
    """Every head width, whole and a part rotated: forward and gradients."""
    for rot, inter in ((d, False), (max(16, d // 32 * 16), True)):
        case = ([33, 0, 5, 1], [4, 0, 90, 1000], 3, 2, d, rot, inter, True, True, {}, 1.0)
        test_forward(nt, case, dtype)
        test_backward(nt, case, dtype)
