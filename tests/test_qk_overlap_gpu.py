"""Outputs of the per-head norm that lie between one another without touching
are no overlap: packed slices, neighbours, in place beside a shared input."""
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


@pytest.mark.parametrize("tokens", [1, 2, 33])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (1, 5)])
def test_packed_outputs_and_a_shared_input(lib, tokens, Hq, Hk):
    L, D = lib, 32
    g = torch.Generator(device=DEV).manual_seed(tokens)
    gamma = torch.randn(2, D, generator=g, device=DEV)
    x = torch.randn(tokens, max(Hq, Hk), D, generator=g, device=DEV)
    q, k = x[:, :Hq], x[:, :Hk]  # one projection for both sides
    want = [R.qk_fw(t, gamma[i], None, None, None, False, 1e-6) for i, t in enumerate((q, k))]

    def halves(buf):  # keys first
        return buf[:, Hk * D:].view(tokens, Hq, D), buf[:, :Hk * D].view(tokens, Hk, D)

    qo, ko = halves(torch.empty(tokens, (Hq + Hk) * D, device=DEV))
    out = L.qk_norm_rope_fw(q, k, gamma[0], gamma[1], q_out=qo, k_out=ko)
    for y, (w, _) in zip(out[:2], want):
        R.check(y, *w, "packed")
    flat = torch.empty(tokens * (Hq + Hk) * D, device=DEV)  # one right behind the other
    n = tokens * Hq * D
    out = L.qk_norm_rope_fw(q, k, gamma[0], gamma[1], q_out=flat[:n].view(tokens, Hq, D),
                            k_out=flat[n:].view(tokens, Hk, D))
    for y, (w, _) in zip(out[:2], want):
        R.check(y, *w, "end to end")
    qi, ki = halves(torch.randn(tokens, (Hq + Hk) * D, generator=g, device=DEV))
    dq, dk = qi.clone(), ki.clone()
    wb = [R.qk_bw(d, t, gamma[i], out[2 + i], None, None, None, False)
          for i, (d, t) in enumerate(((dq, q), (dk, k)))]
    got = L.qk_norm_rope_bw(qi, ki, q, k, gamma[0], gamma[1], out[2], out[3], dq=qi, dk=ki)
    for i in range(2):
        R.check(got[i], *wb[i][0], "packed, in place")
        R.check(got[2 + i], *wb[i][1], "dgamma")
    # both sides in place on one tensor is refused, and nothing is written
    keep = x.clone()
    with pytest.raises(L.LsError, match="overlapping"):
        L.qk_norm_rope_fw(q, k, gamma[0], gamma[1], q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(x, keep)
