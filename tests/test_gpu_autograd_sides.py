"""qk_norm_rope of one side with the other's gamma given as well."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("side", ["q", "k"])
def test_gamma_of_an_absent_side(side):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_batching_gb300 import autograd as ag, build, nt
    build.build()
    x = torch.randn(30, 2, 64, device=DEV, requires_grad=True)
    g, other = (torch.rand(64, device=DEV, requires_grad=True) for _ in range(2))
    turns, pos = nt.nt_rope_turns(64, device=DEV), torch.arange(30, dtype=torch.int32, device=DEV)
    up = torch.randn(30, 2, 64, device=DEV)

    def run(other):
        if side == "q":
            out = ag.qk_norm_rope(x, None, turns, positions=pos, q_gamma=g, k_gamma=other)[0]
        else:
            out = ag.qk_norm_rope(None, x, turns, positions=pos, q_gamma=other, k_gamma=g)[1]
        return (out,) + torch.autograd.grad(out, (x, g), up, retain_graph=True), out

    want, _ = run(None)
    got, out = run(other)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.autograd.grad(out, other, up, allow_unused=True)[0] is None
