"""The attention-path operators as they are used together: a training step
(norm and positions, varlen attention, gradients), and serving (prefill by
varlen attention, then one token at a time over the paged cache, with forks,
frees and compaction on the way)."""
import math
import os

import numpy as np
import pytest
import torch

from _attn_path import inv_freq, positions_of, rope
from _helpers import TOL, normwise_err, to_np

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_batching_gb300 import autograd, build, nt as ntmod, paged
    build.build()
    return ntmod, autograd, paged


def _cu(segs):
    return torch.tensor(np.concatenate([[0], np.cumsum(segs)]).astype(np.int32), device=DEV)


def _plain_rope(x, g, pos, freq):
    """The plain form in fp64 torch operations, differentiable."""
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * g
    t = pos.double()[:, None, None] * freq
    h = freq.numel()
    a, b, rest = y[..., :h], y[..., h:2 * h], y[..., 2 * h:]
    return torch.cat((a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos(), rest), -1)


@pytest.mark.parametrize("dtype,name", [(BF, "bf16"), (F32, "f32")])
def test_training_step(mods, dtype, name):
    """Gradients of q, k, v and both gammas through the norm, the positions
    and causal varlen attention, against fp64 autograd of the plain form.  q
    and k are slices of one projection, as a model has them."""
    nt, ag, _ = mods
    segs, H, d = [5, 1, 130, 64], 2, 64
    T = sum(segs)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(T, 3 * H, d, generator=gen).to(dtype)
    gq, gk = (1 + 0.1 * torch.randn(d, generator=gen) for _ in range(2))
    d_o = torch.randn(T, H, d, generator=gen).to(dtype)
    xl, gql, gkl = (t.to(DEV).requires_grad_(True) for t in (x, gq, gk))
    turns = nt.nt_rope_turns(d, device=DEV)
    cu = _cu(segs)
    q, k = ag.qk_norm_rope(xl[:, :H], xl[:, H:2 * H], turns, cu_seqlens=cu, q_gamma=gql, k_gamma=gkl)
    o = ag.varlen_attention(q, k, xl[:, 2 * H:].contiguous(), cu, max(segs), causal=True)
    o.backward(d_o.to(DEV))
    nt.nt_device_status()

    xr, gqr, gkr = (t.double().requires_grad_(True) for t in (x, gq, gk))
    pos, freq = positions_of(segs), inv_freq(d)
    qr, kr = _plain_rope(xr[:, :H], gqr, pos, freq), _plain_rope(xr[:, H:2 * H], gkr, pos, freq)
    outs, r = [], 0
    for n in segs:
        s = torch.einsum("qhd,khd->hqk", qr[r:r + n], kr[r:r + n]) / math.sqrt(d)
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), float("-inf"))
        outs.append(torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), xr[r:r + n, 2 * H:]))
        r += n
    ref = torch.cat(outs)
    ref.backward(d_o.double())
    assert normwise_err(to_np(o), ref.detach().numpy(), dtype=name) <= TOL[name]
    for got, want in ((xl, xr), (gql, gqr), (gkl, gkr)):
        assert got.grad.dtype == got.dtype
        assert normwise_err(to_np(got.grad), want.grad.numpy(), dtype=name) <= TOL[name]


def test_autograd_equals_the_calls(mods):
    """The Function's outputs and gradients are the calls', bit for bit; an
    output that is not used back-propagates zeros; a transposed upstream
    gradient is taken."""
    nt, ag, _ = mods
    T, H, d = 33, 3, 64
    q = torch.randn(T, H, d, device=DEV, dtype=BF, requires_grad=True)
    k = torch.randn(T, H, d, device=DEV, dtype=BF, requires_grad=True)
    g = torch.ones(d, device=DEV, requires_grad=True)
    turns, cu = nt.nt_rope_turns(32, device=DEV), _cu([30, 3])
    qo, ko = ag.qk_norm_rope(q, k, turns, cu_seqlens=cu, q_gamma=g, interleaved=True)
    up = torch.randn(H, T, d, device=DEV, dtype=BF).transpose(0, 1)
    dq, dg = torch.autograd.grad(qo, (q, g), up, retain_graph=True)
    want = nt.nt_qk_norm_rope_bwd(up.contiguous(), torch.zeros_like(k), turns, q=q.detach(), cu_seqlens=cu,
                                  q_gamma=g.detach(), interleaved=True)
    assert torch.equal(dq, want[0]) and torch.equal(dg, want[2])
    assert int(torch.count_nonzero(torch.autograd.grad(qo.sum(), k)[0])) == 0


def test_training_step_captured(mods):
    """Forward and backward captured into one graph and replayed on new
    inputs give what eager calls give."""
    nt, ag, _ = mods
    segs, H, d = [40, 24], 2, 64
    cu, turns = _cu(segs), nt.nt_rope_turns(d, device=DEV)
    q, k, v, up = (torch.randn(64, H, d, device=DEV, dtype=BF) for _ in range(4))
    g = torch.ones(d, device=DEV)

    def step():
        leaves = [t.detach().requires_grad_(True) for t in (q, k, v, g)]
        a, b = ag.qk_norm_rope(leaves[0], leaves[1], turns, cu_seqlens=cu, q_gamma=leaves[3])
        o = ag.varlen_attention(a, b, leaves[2], cu, max(segs), causal=True)
        return (o,) + torch.autograd.grad(o, leaves, up)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for t in (q, k, v, up):
        t.normal_()
    graph.replay()
    got = [t.clone() for t in outs]
    want = step()
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a, b)
    for a, b in zip(got[2:], want[2:]):
        assert normwise_err(to_np(a), to_np(b), dtype="bf16") <= TOL["bf16"]


@pytest.mark.parametrize("dtype,name", [(BF, "bf16"), (F32, "f32")])
@pytest.mark.parametrize("Hk,page", [(4, 16), (2, 24), (1, 5)])
def test_prefill_then_decode(mods, dtype, name, Hk, page):
    """A batch is prefilled and answers token by token; one sequence is
    forked, one freed, the pool compacted.  Every decoded token's attention
    output matches fp64 attention over that sequence's whole history."""
    nt, _, paged = mods
    H, d = 4, 64
    gen = torch.Generator().manual_seed(3)
    gq, gk = (1 + 0.1 * torch.randn(d, generator=gen) for _ in range(2))
    turns, freq = nt.nt_rope_turns(d, base=500000.0, device=DEV), inv_freq(d, base=500000.0)
    cache = paged.PagedCache(64, page, Hk, d, dtype=dtype, device=DEV)
    history = {}                                   # of each sequence: rows (q, k, v) of every token

    def project(n):
        return [torch.randn(n, h, d, generator=gen).to(dtype) for h in (H, Hk, Hk)]

    def run(seqs, counts):
        """One step: new tokens normed, turned and written; returns the step
        and the turned queries."""
        new = [project(n) for n in counts]
        for s, rows in zip(seqs, new):
            old = history.get(s, [t[:0] for t in rows])
            history[s] = [torch.cat((a, b)) for a, b in zip(old, rows)]
        q, k, v = (torch.cat([n[i] for n in new]).to(DEV) for i in range(3))
        step = cache.step(seqs, counts)
        q, k = nt.nt_qk_norm_rope(q, k, turns, cu_seqlens=step.cu_seqlens, pos0=step.pos0, q_gamma=gq.to(DEV),
                                  k_gamma=gk.to(DEV))
        cache.write(step, k, v)
        return step, q, k, v

    def reference(s):
        q, k, v = history[s]
        pos = torch.arange(q.shape[0])
        qr, kr = rope(q, pos, freq, gq)[0][-1], rope(k, pos, freq, gk)[0]
        out = []
        for h in range(H):
            j = h // (H // Hk)
            out.append(torch.softmax(kr[:, j] @ qr[h] / math.sqrt(d), 0) @ v[:, j].double())
        return torch.stack(out)

    def decode(seqs):
        step, q, _, _ = run(seqs, [1] * len(seqs))
        o = cache.attend(step, q)
        for i, s in enumerate(seqs):
            assert normwise_err(to_np(o[i]), reference(s).numpy(), dtype=name) <= TOL[name], s

    seqs = [cache.add() for _ in range(4)]
    lens = [37, 1, 80, 16]
    step, q, k, v = run(seqs, lens)
    if Hk == H:                                    # the prefill's own attention, causal and packed
        o, _ = nt.nt_varlen_attn_qk(q, k, v, step.cu_seqlens, step.cu_seqlens, step.max_new, causal=True)
        for s, end in zip(seqs, np.cumsum(lens)):
            assert normwise_err(to_np(o[int(end) - 1]), reference(s).numpy(), dtype=name) <= TOL[name]
    decode(seqs)
    twin = cache.fork(seqs[0])
    history[twin] = [t.clone() for t in history[seqs[0]]]
    decode(seqs + [twin])                          # both write behind the shared part
    cache.free(seqs[2])
    cache.compact()
    late = cache.add()
    run([late, seqs[1]], [7, 20])                  # a mixed prefill: a new sequence and a continued one
    for _ in range(3):
        decode([twin, seqs[3], late, seqs[0], seqs[1]])
    nt.nt_device_status()


def test_first_call_of_a_thread(mods):
    """A host thread whose first CUDA work is a call of the library (as
    autograd's backward thread may be): its tensor maps are encoded all the
    same."""
    import threading
    nt, _, _ = mods
    q, k, v, do = (torch.randn(64, 2, 64, device=DEV, dtype=BF) for _ in range(4))
    cu = _cu([40, 24])
    o, lse = nt.nt_varlen_attn_qk(q, k, v, cu, cu, 40, want_lse=True)
    want = nt.nt_varlen_attn_bwd(q, k, v, o, do, lse, cu, None, 40)
    pages = nt.KVPages(torch.randn(4, 2, 16, 64, device=DEV, dtype=BF), torch.randn(4, 2, 16, 64, device=DEV, dtype=BF))
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    n = torch.tensor([50], dtype=torch.int32, device=DEV)
    paged_want = nt.nt_paged_attn(pages, q[:1], table, n)[0]
    torch.cuda.synchronize()
    for call, ref in ((lambda: nt.nt_varlen_attn_bwd(q, k, v, o, do, lse, cu, None, 40), want),
                      (lambda: nt.nt_paged_attn(pages, q[:1], table, n)[:1], (paged_want,))):
        got = []
        t = threading.Thread(target=lambda: got.append(call()))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert got and all(torch.equal(a, b) for a, b in zip(got[0], ref))


def test_cache_full(mods):
    nt, _, paged = mods
    cache = paged.PagedCache(3, 4, 1, 32, device=DEV)
    a, b = cache.add(), cache.add()
    cache.step([a], [9])
    with pytest.raises(paged.OutOfPages):
        cache.step([b], [1])
    cache.free(a)
    cache.step([b], [12])


def test_one_side_alone(mods):
    """Queries without keys through autograd: the gradients of the call with both."""
    nt, ag, _ = mods
    q, k = (torch.randn(50, h, 64, device=DEV, dtype=BF, requires_grad=True) for h in (4, 2))
    g = torch.rand(64, device=DEV, requires_grad=True)
    turns, cu, up = nt.nt_rope_turns(64, device=DEV), _cu([20, 30]), torch.randn(50, 4, 64, device=DEV, dtype=BF)
    alone, none = ag.qk_norm_rope(q, None, turns, cu_seqlens=cu, q_gamma=g)
    assert none is None
    got = torch.autograd.grad(alone, (q, g), up)
    both = ag.qk_norm_rope(q, k, turns, cu_seqlens=cu, q_gamma=g, k_gamma=g.detach())[0]
    assert torch.equal(alone, both)
    want = torch.autograd.grad(both, (q, g), up)
    assert torch.equal(got[0], want[0])
    # the gammas' sums run over the rows in another order: T H roundings of the sum of magnitudes at most
    y = torch.nn.functional.rms_norm(q.detach().double(), (64,)).abs().amax() * up.double().abs().sum((0, 1)).sum()
    assert float((got[1] - want[1]).abs().max()) <= 200 * 2.0 ** -24 * float(y)


def test_step_is_not_captured(mods):
    _, _, paged = mods
    cache = paged.PagedCache(4, 16, 1, 64, device=DEV)
    a = cache.add()
    x = torch.zeros(1, device=DEV)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        x.add_(1)
        with pytest.raises(RuntimeError):
            cache.step([a], [1])
    assert cache.table.length[a] == 0


def test_cache_on_two_streams(mods):
    """Steps attended to on two streams at once, and in a graph replayed
    beside them, share nothing but the pages."""
    nt, _, paged = mods
    cache = paged.PagedCache(600, 16, 2, 64, device=DEV)
    seqs = [cache.add() for _ in range(4)]
    lens = [4000, 1, 2300, 2600]
    step = cache.step(seqs, lens)
    k, v = (torch.randn(sum(lens), 2, 64, device=DEV, dtype=BF) for _ in range(2))
    cache.write(step, k, v)
    q = [torch.randn(4, 8, 64, device=DEV, dtype=BF) for _ in range(3)]
    want = [cache.attend(step, x) for x in q]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = cache.attend(step, q[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        with torch.cuda.stream(streams[2]):
            graph.replay()
        got = [cache.attend(step, x, stream=s) for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got + [replayed], want + [want[2]]))


def test_first_calls_captured():
    """A process whose first calls of the library are captured ones: what a
    kernel has to be allowed or asked first goes on under a capture."""
    import subprocess
    import sys
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    code = """
import torch
from variable_length_batching_gb300 import nt
D, B = "cuda", torch.bfloat16
pages = nt.KVPages(torch.randn(640, 2, 16, 64, device=D, dtype=B), torch.randn(640, 2, 16, 64, device=D, dtype=B))
q, k = torch.randn(3, 8, 64, device=D, dtype=B), torch.randn(3, 2, 64, device=D, dtype=B)
turns, gamma = nt.nt_rope_turns(64, device=D), torch.ones(64, device=D)
cu, one = (torch.tensor(x, dtype=torch.int32, device=D) for x in ([0, 1, 2, 3], [700, 30, 0]))
tables = [torch.arange(3 * w, dtype=torch.int32, device=D).reshape(3, w) % 640 for w in (2, 50, 12500)]

def step():
    a, b = nt.nt_qk_norm_rope(q, k, turns, cu_seqlens=cu, pos0=one, q_gamma=gamma, k_gamma=gamma)
    g = nt.nt_qk_norm_rope_bwd(a, b, turns, q=q, k=k, cu_seqlens=cu, pos0=one, q_gamma=gamma, k_gamma=gamma)
    o = [nt.nt_paged_attn(pages, a, t, one.clamp(max=16 * t.shape[1]), want_lse=True) for t in tables]
    return [a, b, *g] + [x for y in o for x in y]

s = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=s):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, step()))
nt.nt_device_status()
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads(mods):
    """Calls from two host threads at once, each on a stream of its own."""
    import threading
    nt, _, _ = mods
    pages = nt.KVPages(*(torch.randn(300, 2, 16, 64, device=DEV, dtype=BF) for _ in range(2)))
    table = torch.arange(300, dtype=torch.int32, device=DEV).reshape(3, 100)
    q = torch.randn(3, 8, 64, device=DEV, dtype=BF)
    turns, cu = nt.nt_rope_turns(64, device=DEV), _cu([1, 1, 1])
    lens = torch.tensor([1600, 3, 700], dtype=torch.int32, device=DEV)

    def step(stream=None):
        a, _ = nt.nt_qk_norm_rope(q, None, turns, cu_seqlens=cu, pos0=lens, stream=stream)
        return a, nt.nt_paged_attn(pages, a, table, lens, stream=stream)[0]

    want = step()
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(200):
                got = step(s)
                if not all(torch.equal(x, y) for x, y in zip(got, want)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    nt.nt_device_status()
    assert not bad
