"""The per-head norm's backward with heads on one side only: the other side's
gamma gradient is zero, in a buffer of the caller's too."""
import pytest
import torch

import _position_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transformer_reduce_gb300 import build
    build.build()
    import transformer_reduce_gb300 as L
    L.load()
    return L


@pytest.mark.parametrize("tokens", [0, 13])
@pytest.mark.parametrize("Hq,Hk", [(3, 0), (0, 2), (0, 0)])
@pytest.mark.parametrize("D", [32, 33])
def test_gamma_gradient_of_a_side_without_heads_is_zero(lib, tokens, Hq, Hk, D):
    L = lib
    g = torch.Generator(device=DEV).manual_seed(4)
    q, k, dq, dk = (torch.randn(tokens, h, D, generator=g, device=DEV) for h in (Hq, Hk, Hq, Hk))
    gamma = torch.randn(2, D, generator=g, device=DEV)
    rq, rk = (torch.rand(tokens, h, generator=g, device=DEV) for h in (Hq, Hk))
    given = torch.full((2, D), 7.0, device=DEV)
    got = L.qk_norm_rope_bw(dq, dk, q, k, gamma[0], gamma[1], rq, rk, dgamma_q=given[0],
                            dgamma_k=given[1])
    assert got[2].data_ptr() == given.data_ptr()
    made = L.qk_norm_rope_bw(dq, dk, q, k, gamma[0], gamma[1], rq, rk)
    for i, (d, x, r, h) in enumerate(((dq, q, rq, Hq), (dk, k, rk, Hk))):
        if h and tokens:
            (_, _), (w, t) = R.qk_bw(d, x, gamma[i], r, None, None, None, False)
            R.check(given[i], w, t, "dgamma")
        else:
            assert torch.all(given[i] == 0)
        assert torch.equal(given[i], made[2 + i])
