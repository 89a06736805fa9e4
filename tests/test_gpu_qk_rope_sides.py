"""The backward of the query/key norm keeps the sides apart: what is in q's
rows, NaN and infinities too, does not reach k's gradients, and rows that the
offsets place in no segment reach no gamma's."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def nt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_batching_gb300 import build, nt as ntmod
    build.build()
    return ntmod


# T, H, Hk, d: token counts that leave the last group of tokens part empty
# (4, 8 or 16 tokens a step), head counts that leave a step's second row
# empty, and enough of both that warps go from q's units to k's.
SHAPES = [(4097, 32, 8, 128), (4099, 32, 7, 128), (20001, 9, 1, 32), (30003, 5, 3, 64), (50001, 7, 3, 16),
          (9001, 12, 5, 80), (5003, 6, 3, 256), (9, 3, 1, 32)]


def _tokens(T, H, d, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(T, H, d, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("q_norm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,Hk,d", SHAPES)
def test_bad_queries_leave_the_keys_gradients(nt, T, H, Hk, d, dtype, q_norm, bad):
    """Every query and its upstream gradient NaN or infinite: dk and dk_gamma
    are, bit for bit, those of finite ones."""
    q, k = _tokens(T, H, d, dtype, 1), _tokens(T, Hk, d, dtype, 2)
    uq, uk = _tokens(T, H, d, dtype, 3), _tokens(T, Hk, d, dtype, 4)
    g = torch.ones(d, device=DEV)
    turns = nt.nt_rope_turns(16, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    call = lambda u, x: nt.nt_qk_norm_rope_bwd(u, uk, turns, q=x if q_norm else None, k=k, positions=pos,
                                               q_gamma=g if q_norm else None, k_gamma=g)
    want = call(uq, q)
    got = call(torch.full_like(uq, bad), torch.full_like(q, bad))
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[3], want[3])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unplaced_rows_leave_the_gammas_gradients(nt, dtype):
    """Tokens behind the last segment are flagged and add nothing, whatever
    they hold."""
    T, H, d, end = 70, 3, 64, 50
    x, u = _tokens(T, H, d, dtype, 1), _tokens(T, H, d, dtype, 2)
    g = torch.ones(d, device=DEV)
    turns = nt.nt_rope_turns(d, device=DEV)
    cu = torch.tensor([0, 20, end], dtype=torch.int32, device=DEV)

    def run():
        out = nt.nt_qk_norm_rope_bwd(u, None, turns, q=x, cu_seqlens=cu, q_gamma=g)
        with pytest.raises(nt.NTError):
            nt.nt_device_status()
        return out

    want = run()
    x[end:] = math.nan
    u[end:] = math.inf
    got = run()
    assert torch.equal(got[0][:end], want[0][:end]) and torch.equal(got[2], want[2])
