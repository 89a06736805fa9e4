"""The autograd Functions around the library's calls, without a GPU: the calls
are stood in for by torch operations on detached tensors, as opaque to
autograd as the library's are."""
import pytest
import torch

from variable_length_batching_gb300 import autograd as ag


@pytest.fixture
def rope(monkeypatch):
    """y = x^2 gamma for either side in place of the norm and rotation."""
    def fwd(q, k, turns, q_gamma=None, k_gamma=None, **_):
        one = lambda x, g: None if x is None else x.detach() ** 2 * (1 if g is None else g.detach())
        return one(q, q_gamma), one(k, k_gamma)

    def bwd(uq, uk, turns, q=None, k=None, q_gamma=None, k_gamma=None, **_):
        def one(u, x, g):
            if g is not None and (u is None or x is None):
                raise ValueError("a norm needs its side and its upstream gradient")      # as the library does
            if u is None or g is None:
                return None if u is None else u.detach().clone(), None
            u, x, g = (t.detach() for t in (u, x, g))
            return 2 * u * x * g, (u * x * x).sum((0, 1))
        (dq, dqg), (dk, dkg) = one(uq, q, q_gamma), one(uk, k, k_gamma)
        return dq, dk, dqg, dkg

    monkeypatch.setattr(ag.nt, "nt_qk_norm_rope", fwd)
    monkeypatch.setattr(ag.nt, "nt_qk_norm_rope_bwd", bwd)


def _leaves():
    gen = torch.Generator().manual_seed(1)
    q, k = (torch.randn(5, h, 8, generator=gen, requires_grad=True) for h in (2, 1))
    return q, k, torch.rand(8, generator=gen, requires_grad=True)


@pytest.mark.parametrize("upstream", ["constant", "of the outputs", "a leaf"])
def test_second_derivatives_of_rope_raise(rope, upstream):
    q, k, g = _leaves()
    qo, ko = ag.qk_norm_rope(q, k, None, q_gamma=g, k_gamma=g)
    if upstream == "constant":
        grads = torch.autograd.grad(qo.sum() + ko.sum(), (q, k, g), create_graph=True)
    elif upstream == "of the outputs":
        grads = torch.autograd.grad((qo ** 2).sum() + (ko ** 2).sum(), (q, k, g), create_graph=True)
    else:
        u = torch.ones_like(qo, requires_grad=True)
        grads = torch.autograd.grad(qo, (q, g), u, create_graph=True)
    for x in grads:
        with pytest.raises(RuntimeError, match="first derivatives only"):
            ((x ** 2).sum() + (q ** 2).sum()).backward(retain_graph=True)


def test_second_derivatives_without_a_norm_raise_too(rope):
    """Linear in q, but the upstream gradient's derivative would be lost."""
    q, k, _ = _leaves()
    qo, _ = ag.qk_norm_rope(q, k, None)
    dq, = torch.autograd.grad((qo ** 2).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        dq.sum().backward()


def test_first_derivatives_with_create_graph(rope):
    """The graph may be asked for as long as nobody differentiates it."""
    q, k, g = _leaves()
    run = lambda **kw: torch.autograd.grad(sum((y ** 2).sum() for y in ag.qk_norm_rope(q, k, None, q_gamma=g)),
                                           (q, k, g), **kw)
    for a, b in zip(run(create_graph=True), run()):
        assert torch.equal(a, b) and a.requires_grad and not b.requires_grad


def test_second_derivatives_of_varlen_attention_raise(monkeypatch):
    monkeypatch.setattr(ag.nt, "nt_varlen_attn_qk", lambda q, k, v, *a, **kw: (q.detach() * k * v, q.detach().sum(-1)))
    monkeypatch.setattr(ag.nt, "nt_varlen_attn_bwd",
                        lambda q, k, v, o, d_o, *a, **kw: tuple(t.detach() * d_o.detach() for t in (k * v, q * v, q * k)))
    q, k, v = (torch.randn(5, 2, 8, requires_grad=True) for _ in range(3))
    run = lambda **kw: torch.autograd.grad(ag.varlen_attention(q, k, v, torch.tensor([0, 5]), 5).sum(), (q, k, v), **kw)
    for x in run(create_graph=True):
        with pytest.raises(RuntimeError, match="first derivatives only"):
            x.sum().backward(retain_graph=True)
    assert all(not x.requires_grad for x in run())


def test_second_derivatives_of_the_block_raise(monkeypatch):
    names = ("ds", "dW_a", "dW_b", "dgamma", "dbeta", "dW1", "db1", "dW2", "db2", "dW_g", "db_g")
    monkeypatch.setattr(ag.nt, "block_forward", lambda part, s, w, ln_eps: (s.detach() * 2, s.detach(), s.detach() * 3))
    monkeypatch.setattr(ag.nt, "nt_pair_block_backward",
                        lambda *a, **kw: {n: torch.ones(4, 4) for n in names})
    w = [torch.ones(4, 4, requires_grad=True) for _ in names]
    w[6] = None                                                   # no b1
    run = lambda **kw: torch.autograd.grad(sum(y.sum() for y in ag.pair_block(None, *w)), [t for t in w if t is not None],
                                           **kw)
    for x in run(create_graph=True):
        with pytest.raises(RuntimeError, match="first derivatives only"):
            x.sum().backward(retain_graph=True)
    assert all(not x.requires_grad for x in run())


def test_gradients_with_create_graph_can_be_changed_in_place(rope):
    """As those of torch's own operations can: scaled, accumulated, clipped."""
    q, k, g = _leaves()
    loss = lambda: sum((y ** 2).sum() for y in ag.qk_norm_rope(q, k, None, q_gamma=g))
    want = [2 * x for x in torch.autograd.grad(loss(), (q, k, g))]
    grads = torch.autograd.grad(loss(), (q, k, g), create_graph=True)
    for x, y in zip(grads, want):
        assert torch.equal(x.mul_(2), y)
    with torch.no_grad():
        for x, y in zip(grads, want):
            assert torch.equal(x.mul_(0.5).mul_(2), y)
    for _ in range(2):
        loss().backward(create_graph=True)
    for x, y in zip((q, k, g), want):
        assert torch.allclose(x.grad, y)


@pytest.mark.parametrize("side", [0, 1])
def test_a_gamma_without_its_side_takes_no_part(rope, side):
    x, _, g = _leaves()
    other = torch.rand(8, requires_grad=True)
    gammas = (g, other) if side == 0 else (other, g)
    out = ag.qk_norm_rope(*((x, None) if side == 0 else (None, x)), None, q_gamma=gammas[0], k_gamma=gammas[1])[side]
    dx, dg, none = torch.autograd.grad(out.sum(), (x, g, other), allow_unused=True)
    assert none is None and torch.equal(dx, (2 * x * g).detach()) and dg is not None
